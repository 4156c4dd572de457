// Attention of a few queries per head over the 8-bit paged cache on gfx950.
//
// For every (sequence, KV head) the G query heads' W queries form the R = G*W
// rows of two products against the same keys and values:
//   s = c * ks * <q, code_k>, p = 2^(s - m), l = sum p, out = sum p * vs * code_v / l
// with c = scale * log2(e), ks and vs the page scales, m a running maximum.
// Each cached byte is read once for all R rows; with the few rows of a decode
// step the bound is HBM: 2*d bytes per key.
//
// Both products run on fp16 matrix instructions, 16x16x32: e4m3 and int8 codes
// are exact in fp16, so is a bf16 query scaled by a power of two (elements
// below 2^-29 of the row's largest lose bits), and the weights keep 11 bits.
// A weight carries its page's value scale, w = 2^(s + log2 vs - m2) with a
// maximum m2 of its own, so that it stays in (0, 1] whatever the scales are.
//
// Both products are taken transposed, S' = K Q' and O' = V' P': the lane that
// holds eight scores of a query row (keys 4g..4g+3 of two 16-key tiles, g its
// 16-lane group) holds exactly the eight weights that the second product wants
// from it, so the weights never leave their lane.  K fragments are loaded as
// they lie in memory; V is read eight keys deep and D/16 values wide per lane
// and turned in registers by byte permutes.
//
// The keys of a head are cut into pieces by its own length (q8_chunk); the
// four waves of a workgroup take the 32-key tiles of a piece in turn, and
// their sums meet in LDS.  A second kernel joins the pieces where there are
// several.
#include "kvc_q8.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kMaxChunk = 2048;
constexpr uint32_t kNone = 0xffffffffu;  // no row: past the end or in no page

struct Args {
  Q8 c;
  int W, R, pieces;  // pieces: of the longest length, the grid's
  int n0;            // first head of this launch
  float c_log2;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part;  // [n][row][piece][D] sums, then [n][row][piece][4] (m, l, m2, -)
  float* stat;
};

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Codes 2*HI and 2*HI+1 of w as fp16.
template <int FMT, bool HI>
__device__ __forceinline__ f16x2 pair(uint32_t w) {
  if constexpr (FMT == KVC_Q8_E4M3) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
  } else {
    // 0x6400 + b is 1024 + b in fp16; b = code + 128
    const uint32_t h = __builtin_amdgcn_perm(0x64646464u, w, HI ? 0x04030402u : 0x04010400u);
    return __builtin_bit_cast(f16x2, h) - f16x2{_Float16(1152), _Float16(1152)};
  }
}

// Eight codes (two words) as a matrix fragment.
template <int FMT>
__device__ __forceinline__ f16x8 frag(uint32_t a, uint32_t b) {
  if constexpr (FMT == KVC_Q8_INT8) a ^= 0x80808080u, b ^= 0x80808080u;
  const f16x2 x = pair<FMT, false>(a), y = pair<FMT, true>(a), z = pair<FMT, false>(b),
              w = pair<FMT, true>(b);
  return f16x8{x.x, x.y, y.x, y.y, z.x, z.y, w.x, w.y};
}

// 4x4 byte transpose: word i of the result holds byte i of the four inputs.
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t* o) {
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u);  // a0 b0 a1 b1
  const uint32_t ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);  // a2 b2 a3 b3
  const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

// One output value from its sums: the weights were relative to 2^m2 and carried
// the value scales, l is relative to 2^m.
__device__ __forceinline__ void finish(const Args& A, size_t row, int D, int dim, float sum,
                                       float l, float m, float m2) {
  A.out[row * D + dim] = to_bf16(l == 0.0f ? 0.0f : sum * (fast_exp2(m2 - m) / l));
  if (A.lse && dim == 0)
    A.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

template <int D, int FMT, int MT>
__global__ __launch_bounds__(kThreads) void k_q8_attend(Args A) {
  constexpr int kSteps = D / 32;        // matrix steps over the head dimension
  constexpr int kTiles = D / 16;        // 16-value tiles of the output
  constexpr int kVWords = D / 64;       // words of one key's values in a lane
  constexpr int kRowF = D + 4;          // floats of one merged row: sums, m, l, m2
  constexpr int kKeysLds = kMaxChunk * 3;
  constexpr int kMergeLds = 4 * 16 * kRowF;
  __shared__ __align__(16) float lds[kKeysLds > kMergeLds ? kKeysLds : kMergeLds];
  uint32_t* const row_of = reinterpret_cast<uint32_t*>(lds);  // pool row of each key
  float* const ks_of = lds + kMaxChunk;                       // its key scale
  float* const lv_of = lds + 2 * kMaxChunk;                   // log2 of its value scale

  const Q8& c = A.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int piece = int(blockIdx.x % unsigned(A.pieces));
  const int n = A.n0 + int(blockIdx.x / unsigned(A.pieces)), rb = blockIdx.y;
  const int b = n / c.H, h = n % c.H;
  const int len = q8_len(c, b);
  const int chunk = q8_chunk(len);
  const int t0 = piece * chunk;
  if (t0 >= len && piece > 0) return;
  const int keys = len - t0 < chunk ? len - t0 : chunk;  // of this piece, 0 for an empty sequence
  const bool alone = len <= chunk;

  // Where the keys of this piece are.
  const int padded = (keys + 31) & ~31;
  for (int i = tid; i < padded; i += kThreads) {
    uint32_t row = kNone;
    float ks = 0.0f, lv = -INFINITY;
    if (i < keys) {
      const uint32_t t = uint32_t(t0 + i), j = quot(c.div, t);
      const int page = q8_page(c, b, int(j));
      if (page >= 0) {
        const uint32_t ph = uint32_t(page) * uint32_t(c.H) + uint32_t(h);
        row = ph * c.div.d + (t - j * c.div.d);
        ks = c.ks[ph];
        lv = __builtin_amdgcn_logf(c.vs[ph]);
      }
    }
    row_of[i] = row;
    ks_of[i] = ks;
    lv_of[i] = lv;
  }

  // Queries: fp16 fragments of rows scaled by a power of two.
  f16x8 qf[MT][kSteps];
  float qc[MT];
  int last[MT];  // last key this row attends to
  float m[MT], m2[MT], l[MT];
  f32x4 acc[MT][kTiles];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = (rb * MT + mt) * 16 + col;
    u32x4 raw[kSteps];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      raw[s] = u32x4{0, 0, 0, 0};
      if (r < A.R) {
        const int dim = (s >> 1) * 64 + g * 16 + (s & 1) * 8;
        raw[s] = *reinterpret_cast<const u32x4*>(A.q + (size_t(n) * A.R + r) * D + dim);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = raw[s][i] & 0x7fffu, hi = (raw[s][i] >> 16) & 0x7fffu;
        top = top > lo ? top : lo;
        top = top > hi ? top : hi;
      }
    }
#pragma unroll
    for (int off = 16; off <= 32; off <<= 1) {
      const uint32_t o = uint32_t(__shfl_xor(int(top), off));
      top = top > o ? top : o;
    }
    int up = 14 - (int(top >> 7) - 127);  // largest magnitude to [2^14, 2^15)
    up = up > 126 ? 126 : up;
    const float mul = __uint_as_float(uint32_t(up + 127) << 23);
    qc[mt] = A.c_log2 * __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[mt][s][2 * i] = _Float16(__uint_as_float(raw[s][i] << 16) * mul);
        qf[mt][s][2 * i + 1] = _Float16(__uint_as_float(raw[s][i] & 0xffff0000u) * mul);
      }
    last[mt] = r < A.R ? len - A.W + r % A.W - t0 : -1;
    m[mt] = m2[mt] = -INFINITY;
    l[mt] = 0.0f;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[mt][i] = f32x4{0, 0, 0, 0};
  }
  __syncthreads();

  for (int tile = wave * 32; tile < keys; tile += 128) {
    // K fragments of two 16-key tiles, as they lie.
    f16x8 kf[2][kSteps];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t row = row_of[tile + half * 16 + col];
#pragma unroll
      for (int s = 0; s < kSteps; s += 2) {
        u32x4 x = {0, 0, 0, 0};
        if (row != kNone)
          x = *reinterpret_cast<const u32x4*>(c.k + size_t(row) * D + s * 32 + g * 16);
        kf[half][s] = frag<FMT>(x.x, x.y);
        kf[half][s + 1] = frag<FMT>(x.z, x.w);
      }
    }
    // V: this lane's keys are 4g..4g+3 of both tiles, its values D/16 wide.
    const u32x4 rows[2] = {*reinterpret_cast<const u32x4*>(row_of + tile + 4 * g),
                           *reinterpret_cast<const u32x4*>(row_of + tile + 16 + 4 * g)};
    uint32_t vw[8][kVWords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t row = rows[i >> 2][i & 3];
#pragma unroll
      for (int w = 0; w < kVWords; ++w) vw[i][w] = 0;
      if (row != kNone) {
        const uint8_t* at = c.v + size_t(row) * D + col * (D / 16);
        if constexpr (kVWords == 2) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(at);
          vw[i][0] = x.x, vw[i][1] = x.y;
        } else {
          vw[i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
    }
    f16x8 vf[kTiles];
#pragma unroll
    for (int w = 0; w < kVWords; ++w) {
      uint32_t lo[4], hi[4];
      turn4(vw[0][w], vw[1][w], vw[2][w], vw[3][w], lo);
      turn4(vw[4][w], vw[5][w], vw[6][w], vw[7][w], hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) vf[w * 4 + i] = frag<FMT>(lo[i], hi[i]);
    }
    const f32x4 ks[2] = {*reinterpret_cast<const f32x4*>(ks_of + tile + 4 * g),
                         *reinterpret_cast<const f32x4*>(ks_of + tile + 16 + 4 * g)};
    const f32x4 lv[2] = {*reinterpret_cast<const f32x4*>(lv_of + tile + 4 * g),
                         *reinterpret_cast<const f32x4*>(lv_of + tile + 16 + 4 * g)};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float s[8], x[8];
      float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[half][k], qf[mt][k], a, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = half * 4 + i;
          const bool seen = tile + half * 16 + 4 * g + i <= last[mt] && rows[half][i] != kNone;
          s[j] = seen ? a[i] * (ks[half][i] * qc[mt]) : -INFINITY;
          x[j] = s[j] + lv[half][i];
          top = fmaxf(top, s[j]);
          top2 = fmaxf(top2, x[j]);
        }
      }
#pragma unroll
      for (int off = 16; off <= 32; off <<= 1) {
        top = fmaxf(top, __shfl_xor(top, off));
        top2 = fmaxf(top2, __shfl_xor(top2, off));
      }
      if (__any(top > m[mt] || top2 > m2[mt])) {
        const float nm = fmaxf(m[mt], top), nm2 = fmaxf(m2[mt], top2);
        const float f = nm == -INFINITY ? 1.0f : fast_exp2(m[mt] - nm);
        const float f2 = nm2 == -INFINITY ? 1.0f : fast_exp2(m2[mt] - nm2);
        l[mt] *= f;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[mt][i] *= f2;
        m[mt] = nm;
        m2[mt] = nm2;
      }
      const float base = m[mt] == -INFINITY ? 0.0f : m[mt];
      const float base2 = m2[mt] == -INFINITY ? 0.0f : m2[mt];
      f16x8 w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        l[mt] += fast_exp2(s[j] - base);
        w[j] = _Float16(fast_exp2(x[j] - base2));
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i], w, acc[mt][i], 0, 0, 0);
    }
  }

  // The four waves' sums meet in LDS (over the key arrays), 16 rows at a time.
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
#pragma unroll
    for (int off = 16; off <= 32; off <<= 1) l[mt] += __shfl_xor(l[mt], off);
    float* to = lds + (wave * 16 + col) * kRowF;
#pragma unroll
    for (int r = 0; r < 4; ++r)  // values of row 4g + r of tile i: dim (4g + r) * kTiles + i
#pragma unroll
      for (int i = 0; i < kTiles; ++i) to[(4 * g + r) * kTiles + i] = acc[mt][i][r];
    if (g == 0) {
      to[D] = m[mt];
      to[D + 1] = l[mt];
      to[D + 2] = m2[mt];
    }
    __syncthreads();
    const int r0 = (rb * MT + mt) * 16, rows_here = A.R - r0 < 16 ? A.R - r0 : 16;
    for (int e = tid; e < rows_here * D; e += kThreads) {
      const int r = e / D, dim = e % D;
      const float* at = lds + r * kRowF;
      float M = -INFINITY, M2 = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        M = fmaxf(M, at[w * 16 * kRowF + D]);
        M2 = fmaxf(M2, at[w * 16 * kRowF + D + 2]);
      }
      const float base = M == -INFINITY ? 0.0f : M, base2 = M2 == -INFINITY ? 0.0f : M2;
      float sum = 0.0f, L = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float* aw = at + w * 16 * kRowF;
        sum += aw[dim] * fast_exp2(aw[D + 2] - base2);
        L += aw[D + 1] * fast_exp2(aw[D] - base);
      }
      const size_t row = size_t(n) * A.R + r0 + r;
      if (alone) {
        finish(A, row, D, dim, sum, L, base, base2);
      } else {
        const size_t at_piece = row * A.pieces + piece;
        A.part[at_piece * D + dim] = sum;
        if (dim == 0) {
          float* st = A.stat + at_piece * 4;
          st[0] = M, st[1] = L, st[2] = M2;
        }
      }
    }
  }
}

// Joins the pieces of one row.
template <int D>
__global__ __launch_bounds__(D) void k_q8_join(Args A, size_t row0) {
  const size_t row = row0 + blockIdx.x;
  const int b = int(row / A.R / unsigned(A.c.H));
  const int len = q8_len(A.c, b), chunk = q8_chunk(len);
  if (len <= chunk) return;
  const int pieces = (len + chunk - 1) / chunk, dim = threadIdx.x;
  const float* st = A.stat + row * A.pieces * 4;
  const float* part = A.part + row * A.pieces * D + dim;
  float M = -INFINITY, M2 = -INFINITY;
  for (int p = 0; p < pieces; ++p) M = fmaxf(M, st[p * 4]), M2 = fmaxf(M2, st[p * 4 + 2]);
  const float base = M == -INFINITY ? 0.0f : M, base2 = M2 == -INFINITY ? 0.0f : M2;
  float sum = 0.0f, L = 0.0f;
  for (int p = 0; p < pieces; ++p) {
    sum += part[size_t(p) * D] * fast_exp2(st[p * 4 + 2] - base2);
    L += st[p * 4 + 1] * fast_exp2(st[p * 4] - base);
  }
  finish(A, row, D, dim, sum, L, base, base2);
}

template <int D, int FMT, int MT>
void attend(Args A, hipStream_t s) {
  // (head, piece) in x, below 2^23 workgroups (the grid counts work-items in
  // 32 bits), row blocks in y.
  const int heads = A.c.B * A.c.H, blocks_y = (A.R + MT * 16 - 1) / (MT * 16);
  const int most = (1 << 23) / A.pieces;
  for (A.n0 = 0; A.n0 < heads; A.n0 += most) {
    const int nh = heads - A.n0 < most ? heads - A.n0 : most;
    k_q8_attend<D, FMT, MT><<<dim3(unsigned(nh) * unsigned(A.pieces), unsigned(blocks_y)),
                              kThreads, 0, s>>>(A);
  }
  if (A.pieces == 1) return;
  const size_t rows = size_t(heads) * A.R, step = size_t(1) << 23;
  for (size_t r0 = 0; r0 < rows; r0 += step)
    k_q8_join<D><<<unsigned(rows - r0 < step ? rows - r0 : step), D, 0, s>>>(A, r0);
}

template <int D, int FMT>
void attend_rows(const Args& A, hipStream_t s) {
  if (A.R <= 16) attend<D, FMT, 1>(A, s);
  else attend<D, FMT, 2>(A, s);
}

}  // namespace

hipError_t launch_q8_attend(const Q8& c, int G, int W, float c_log2, const void* q, void* out,
                            float* lse, float* part, hipStream_t s) {
  Args A;
  A.c = c;
  A.W = W;
  A.R = G * W;
  A.pieces = q8_max_pieces(c.cap);
  A.n0 = 0;
  A.c_log2 = c_log2;
  A.q = static_cast<const uint16_t*>(q);
  A.out = static_cast<uint16_t*>(out);
  A.lse = lse;
  A.part = part;
  A.stat = part + size_t(c.B) * c.H * A.R * A.pieces * c.D;
  if (c.D == 128 && c.fmt == KVC_Q8_E4M3) attend_rows<128, KVC_Q8_E4M3>(A, s);
  else if (c.D == 128) attend_rows<128, KVC_Q8_INT8>(A, s);
  else if (c.fmt == KVC_Q8_E4M3) attend_rows<64, KVC_Q8_E4M3>(A, s);
  else attend_rows<64, KVC_Q8_INT8>(A, s);
  return hipGetLastError();
}

}  // namespace kvc
