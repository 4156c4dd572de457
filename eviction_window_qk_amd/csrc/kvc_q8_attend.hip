// Attention of a few queries per head over the 8-bit paged cache on gfx950.
//
// For every (sequence, KV head) the G query heads' W queries form the R = G*W
// rows of two products against the same keys and values:
//   x = c * ks * <q, code_k> + log2 r,  w = 2^(x - m),
//   l = sum w / r,  out = top * sum w * code_v / l
// with c = scale * log2(e), ks and vs the page scales, top the largest vs among
// the keys that a workgroup takes and r = vs / top, m kHead to kHead + kSlack below
// the running maximum of x.  Each cached byte is read once for all R rows; with the few rows of a
// decode step the bound is HBM: 2*d bytes per key.
//
// Both products run on fp16 matrix instructions, 16x16x32: e4m3 and int8 codes
// are exact in fp16, so is a bf16 query scaled by a power of two (elements
// below 2^-29 of the row's largest lose bits), and the weights keep 11 bits down to
// 2^-23 of the row's largest, below that a step of 2^-33 of it (bf16 outputs
// need 9).
// A weight carries its page's value scale inside the exponent, so one exp2 a
// score gives a number in (0, 2^15] whatever the scales are; the denominator
// takes the scale out again, in fp32.  The scale is taken relative to the
// largest of the workgroup's keys, and is at least kQuiet: hundreds of zero values
// (scale 2^-126) weigh in the denominator as much as any others, and 2^126 each
// would overflow it.
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
// several.  Where a piece's keys are and what they weigh is looked up once, into
// LDS: for four keys at a time where the page size is a multiple of four (every
// lane's keys come in fours), for each key where it is not.  With short pieces
// the look-up and the merge, not the keys, are what a batch of ordinary lengths
// spends its time on: on 512 heads of 1100 keys 11 of 40 us went into a look-up
// by single keys.
#include <type_traits>

#include "kvc_q8.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kMaxChunk = kQ8MaxChunk;
// What a look-up says of its keys: the first one's row in the pools, the key
// scale, log2 of the value scale (-inf: there is no page) and its reciprocal.
struct __align__(16) Where {
  uint32_t row;
  float ks, lv, iv;
};

// m is set kHead below a row's maximum, and follows once a score is kSlack past that
// maximum: the sums are scaled once or twice a row and wave, not at every new
// maximum (20 rows on ragged drafts 57.6 us, 55.2 so).  Weights reach 2^15, fp16's
// last binade, so that they are whole down to 2^-23 of the largest (2^-14 with m at
// the maximum), where fp16 turns subnormal.
constexpr float kSlack = 6.0f, kHead = 9.0f;
constexpr float kMost = 0x1.fffffep127f;
// A value scale further than kQuiet below the piece's largest (an empty page's)
// counts as kQuiet of it.  The denominator is held in units of kUnit: a key adds at
// most 2^15 / (kUnit kQuiet) = 2^67, so a row that sees quiet keys only stays below
// 2^97 over the 2^30 keys of the longest table.  Sums are scaled by the
// square root of a power of two, twice: in one step the factor would vanish at
// 2^-126 before a quiet key's sum does.  The exp2 of a key vanishes there, and
// takes at most 2^-35 of the row's sum with it.
constexpr float kQuiet = 0x1p-100f;
constexpr float kUnit = 0x1p48f;
constexpr uint32_t kNone = 0xffffffffu;  // no row: past the end or in no page

struct Args {
  Q8 c;
  int W, R, pieces;  // pieces: of the longest length, the grid's
  FastDiv by_W, by_R, by_pieces, by_H, by_blocks;
  int units, unit0;  // (head, piece) pairs of n0's heads, first one of this launch
  int n0;            // first head of this launch
  int lds_rows;      // rows of a wave's sums in LDS: min(R, 16)
  float c_log2;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part;  // [n][row][piece][D] outputs of a piece
  float* stat;  // [n][row][piece][2] their m, l
};

// Largest of eight.  (Written with fmaxf it is eleven instructions: each operand
// that a branch may have changed is quieted first.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float x;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(x) : "v"(a), "v"(b), "v"(c));
  return x;
}
__device__ __forceinline__ float max8(const float (&y)[8]) {
  return max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), max3(y[6], y[7], y[7]));
}

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

template <bool STREAM, class T>
__device__ __forceinline__ T load(const uint8_t* at) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T*>(at));
  else return *reinterpret_cast<const T*>(at);
}

// Maximum over the workgroup, in every thread.
__device__ __forceinline__ float block_max(float x, float* sh) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  x = sh[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) x = fmaxf(x, sh[w]);
  return x;
}

// log2 of a sum in kUnit: multiplied first, an ordinary sum loses no bits to the 48.
__device__ __forceinline__ float log2_sum(float l) {
  return l < 1.0f ? __builtin_amdgcn_logf(l * kUnit) : __builtin_amdgcn_logf(l) + 48.0f;
}

// Four output values of a row, and its sum of weights l (in kUnit) relative to 2^m.
__device__ __forceinline__ void finish(const Args& A, size_t row, int D, int dim, f32x4 out,
                                       float l, float m) {
  *reinterpret_cast<u16x4*>(A.out + row * D + dim) =
      u16x4{to_bf16(out.x), to_bf16(out.y), to_bf16(out.z), to_bf16(out.w)};
  if (A.lse && dim == 0)
    A.lse[row] = l == 0.0f ? -INFINITY : (m + log2_sum(l)) * 0.6931471805599453f;
}

// Four waves a SIMD: a tile of each in flight covers the latency of HBM, and
// nothing is gained by a second tile in registers at two waves (29 against 24 us
// on 256 heads of 1100 keys).  The checks for keys that are not seen sit in a
// branch of the one tile body: a body with and one without them took 160
// registers for 120 and ran at three waves, 10 % slower on ragged drafts.  32 rows
// at D = 128 need the registers of two waves (at three they spill: 146 us
// became 269 on 128 heads of 16384 keys).
// Look-ups of single keys take up to ten registers more: asked for four waves the
// compiler spills some of them where it needs none for three (and four fit, but for
// e4m3 at D = 128 with 130 registers).
constexpr int waves(int D, int FMT, int MT, int GROUP) {
  if (D == 128 && MT == 2) return 2;
  return GROUP == 1 && (D == 128 || (MT == 2 && FMT == KVC_Q8_INT8)) ? 3 : 4;
}
template <int D, int FMT, int MT, int GROUP, bool STREAM>
__global__ __launch_bounds__(kThreads, waves(D, FMT, MT, GROUP)) void k_q8_attend(Args A) {
  constexpr int kSteps = D / 32;        // matrix steps over the head dimension
  constexpr int kTiles = D / 16;        // 16-value tiles of the output
  constexpr int kVWords = D / 64;       // words of one key's values in a lane
  constexpr int kRowF = D + 4;          // floats of one merged row: sums, m, l
  constexpr int kGroups = 4 / GROUP;    // look-ups of four keys
  constexpr int kPerTile = 32 / GROUP;
  extern __shared__ __align__(16) unsigned char lds_raw[];
  Where* const where = reinterpret_cast<Where*>(lds_raw);  // then the waves' sums
  float* const lds = reinterpret_cast<float*>(lds_raw);
  __shared__ float top_of[kWaves];
  __shared__ uint32_t none_of[kMaxChunk / 32];  // which look-ups of a tile found no page

  const Q8& c = A.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  // Pieces of one head together, each head's rotated by one: workgroups go to
  // the XCDs in turn, and where only the first pieces of a long table have keys
  // they would all be one XCD's (512 heads of 128 keys in tables of 16384: 118 us
  // without the rotation, 18 with it).
  // The row blocks of a piece follow each other on one XCD, whose L2 then reads its
  // keys once (81 rows on 9 heads of 62000 keys: 57 us with the blocks in a grid
  // dimension of their own, 52 so).
  const uint32_t eight = quot(A.by_blocks, blockIdx.x >> 3);
  const int rb = int((blockIdx.x >> 3) - eight * A.by_blocks.d);
  const uint32_t unit = uint32_t(A.unit0) + eight * 8 + (blockIdx.x & 7);
  if (unit >= uint32_t(A.units)) return;
  const int nth = int(quot(A.by_pieces, unit));
  int piece = int(unit) - nth * A.pieces + (nth - int(quot(A.by_pieces, uint32_t(nth))) * A.pieces);
  piece -= piece >= A.pieces ? A.pieces : 0;
  const int n = A.n0 + nth;
  const int b = int(quot(A.by_H, uint32_t(n))), h = n - b * c.H;

  const int len = q8_len(c, b);
  const int chunk = q8_chunk(len, A.R);
  const int t0 = piece * chunk;
  if (t0 >= len && piece > 0) return;
  const int keys = len - t0 < chunk ? len - t0 : chunk;  // of this piece, 0 for an empty sequence
  const bool alone = len <= chunk;

  // Queries, on their way while the keys are looked up.
  u32x4 raw[MT][kSteps];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = (rb * MT + mt) * 16 + col;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      raw[mt][s] = u32x4{0, 0, 0, 0};
      if (r < A.R) {
        const int dim = (s >> 1) * 64 + g * 16 + (s & 1) * 8;
        raw[mt][s] = *reinterpret_cast<const u32x4*>(A.q + (size_t(n) * A.R + r) * D + dim);
      }
    }
  }
  // Where the keys of this piece are.  A look-up that finds no page (or lies past
  // the end) points to row 0, whose bytes are dropped later.  The scales follow
  // after a first barrier, when the first tile's loads are on their way.
  const int padded = (keys + 31) & ~31, lookups = padded / GROUP;
  for (int i = tid; i < ((lookups + 63) & ~63); i += kThreads) {
    uint32_t row = kNone;
    if (i * GROUP < keys) {
      const uint32_t t = uint32_t(t0 + i * GROUP), j = quot(c.div, t);
      const int page = q8_page(c, b, int(j));
      if (page >= 0)
        row = (uint32_t(page) * uint32_t(c.H) + uint32_t(h)) * c.div.d + (t - j * c.div.d);
    }
    const uint64_t none = __ballot(row == kNone);
    if (i < lookups) {
      where[i].row = row == kNone ? 0 : row;
      where[i].lv = row == kNone ? -INFINITY : 0.0f;
      if (lane % kPerTile == 0) none_of[i / kPerTile] = uint32_t(none >> lane) & (0xffffffffu >> (32 - kPerTile));
    }
  }
  __syncthreads();

  // One tile of 32 keys as it is loaded.  K: this lane's keys are col of either
  // half, its bytes g*16..; V: keys 4g..4g+3 of both halves, D/16 bytes of each.
  struct Tile {
    u32x4 k[2][kSteps / 2];
    uint32_t v[8][kVWords];
  };
  auto fetch = [&](int tile, Tile& x) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key = tile + half * 16 + col;
      const uint8_t* at = c.k + size_t(where[key / GROUP].row) * D + (col % GROUP * D + g * 16);
#pragma unroll
      for (int s = 0; s < kSteps / 2; ++s) x.k[half][s] = load<STREAM, u32x4>(at + s * 64);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int key = tile + (i >> 2) * 16 + 4 * g + (i & 3);
      const uint8_t* at = c.v + size_t(where[key / GROUP].row) * D + (i % GROUP * D + col * (D / 16));
      if constexpr (kVWords == 2) {
        const u32x2 y = load<STREAM, u32x2>(at);
        x.v[i][0] = y.x, x.v[i][1] = y.y;
      } else {
        x.v[i][0] = load<STREAM, uint32_t>(at);
      }
    }
  };
  Tile cur;
  if (wave * 32 < keys) fetch(wave * 32, cur);

  float vtop = 0.0f;
  for (int i = tid; i < lookups; i += kThreads) {
    float ks = 0.0f, vs = 0.0f;
    if (where[i].lv == 0.0f) {
      const uint32_t ph = quot32(c.div, where[i].row);
      ks = c.ks[ph];
      vs = c.vs[ph];
    }
    where[i].ks = ks;
    where[i].iv = vs;
    vtop = fmaxf(vtop, vs);
  }
  vtop = fmaxf(block_max(vtop, top_of), 0x1p-126f);
  vtop = __uint_as_float(uint32_t(__builtin_amdgcn_readfirstlane(int(__float_as_uint(vtop)))));
  const float by_top = 1.0f / vtop;
  for (int i = tid; i < lookups; i += kThreads) {
    const float r = fmaxf(where[i].iv * by_top, kQuiet);
    if (where[i].lv == 0.0f) where[i].lv = __builtin_amdgcn_logf(r);
    where[i].iv = __builtin_amdgcn_rcpf(r * kUnit);
  }

  // Queries to fp16 fragments of rows scaled by a power of two.
  f16x8 qf[MT][kSteps];
  float qc[MT];
  int last[MT];  // last key this row attends to
  float base[MT], most[MT], l[MT];  // most: -inf until the row has a base
  f32x4 acc[MT][kTiles];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = (rb * MT + mt) * 16 + col;
    u16x2 tops = {0, 0};  // bf16 magnitudes order like their bits
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        tops = __builtin_elementwise_max(
            tops, __builtin_bit_cast(u16x2, raw[mt][s][i] & 0x7fff7fffu));
    uint32_t top = tops.x > tops.y ? tops.x : tops.y;
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
        qf[mt][s][2 * i] = _Float16(__uint_as_float(raw[mt][s][i] << 16) * mul);
        qf[mt][s][2 * i + 1] = _Float16(__uint_as_float(raw[mt][s][i] & 0xffff0000u) * mul);
      }
    last[mt] = r < A.R ? len - A.W + (r - int(quot(A.by_W, uint32_t(r))) * A.W) - t0 : 0x7ffffffe;  // rows that are none: see all
    base[mt] = 0.0f;
    most[mt] = -INFINITY;
    l[mt] = 0.0f;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[mt][i] = f32x4{0, 0, 0, 0};
  }
  const int low = len - A.W - t0;  // the first query's last key: all rows see the keys up to it
  __syncthreads();

  auto work = [&](int tile, Tile& x, bool checked) {
    Where at[2][kGroups];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        at[half][i] = where[(tile + half * 16 + 4 * g) / GROUP + i];
    float scores[MT][8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f16x8 kf[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; s += 2) {
        kf[s] = frag<FMT>(x.k[half][s / 2].x, x.k[half][s / 2].y);
        kf[s + 1] = frag<FMT>(x.k[half][s / 2].z, x.k[half][s / 2].w);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[k], qf[mt][k], a, 0, 0, 0);
        // the scales' product first: one for a look-up's keys, and a tiny query's
        // takes a huge key's back into range
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Where& of = at[half][i / GROUP];
          scores[mt][half * 4 + i] =
              __builtin_fmaf(a[i], fminf(of.ks * qc[mt], kMost), of.lv - base[mt]);
        }
      }
    }
    if (checked) {  // the same for the whole wave
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = tile + (j >> 2) * 16 + 4 * g + (j & 3);
        const bool none = at[j >> 2][(j & 3) / GROUP].lv == -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (t > last[mt] || none) scores[mt][j] = -INFINITY;
#pragma unroll
        for (int u = 0; u < kVWords; ++u)
          if (t >= keys || none) x.v[j][u] = 0;
      }
    }
    // look-ups of single keys: the eight reciprocals come from LDS now, not with
    // the scales above (they would not fit the registers beside them)
    int later = tile + 4 * g;
    if constexpr (GROUP == 1) asm("" : "+v"(later));
    f16x8 w[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float(&y)[8] = scores[mt];
      float top = max8(y);
      if (__any(top > most[mt])) {
#pragma unroll
        for (int off = 16; off <= 32; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
        const float up = top > most[mt] ? top - kHead : 0.0f;
        const float f = most[mt] == -INFINITY ? 1.0f : fast_exp2(-0.5f * up);
        l[mt] = l[mt] * f * f;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[mt][i] *= f * f;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] -= up;
        base[mt] += up;
        most[mt] = top > most[mt] ? kHead + kSlack : most[mt];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = fast_exp2(y[j]);
        const float iv = GROUP == 1 ? where[later + (j >> 2) * 16 + (j & 3)].iv
                                    : at[j >> 2][(j & 3) / GROUP].iv;
        l[mt] = __builtin_fmaf(e, iv, l[mt]);
        w[mt][j] = _Float16(e);
      }
    }
#pragma unroll
    for (int u = 0; u < kVWords; ++u) {
      uint32_t lo[4], hi[4];
      turn4(x.v[0][u], x.v[1][u], x.v[2][u], x.v[3][u], lo);
      turn4(x.v[4][u], x.v[5][u], x.v[6][u], x.v[7][u], hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x8 vf = frag<FMT>(lo[i], hi[i]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          acc[mt][u * 4 + i] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, w[mt], acc[mt][u * 4 + i], 0, 0, 0);
      }
    }
  };
  for (int tile = wave * 32; tile < keys; tile += kWaves * 32) {
    if (tile != wave * 32) fetch(tile, cur);
    work(tile, cur, tile + 31 > low || none_of[tile >> 5] != 0);
  }

  // The waves' sums meet in LDS (over the key arrays), 16 rows at a time.
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
#pragma unroll
    for (int off = 16; off <= 32; off <<= 1) l[mt] += __shfl_xor(l[mt], off);
    const int r0 = (rb * MT + mt) * 16, rows_here = A.R - r0 < 16 ? A.R - r0 : 16;
    float* to = lds + (wave * A.lds_rows + col) * kRowF;
    if (col < rows_here) {
#pragma unroll
      for (int r = 0; r < 4; ++r)  // values of row 4g + r of tile i: dim (4g + r) * kTiles + i
#pragma unroll
        for (int i = 0; i < kTiles; ++i) to[(4 * g + r) * kTiles + i] = acc[mt][i][r];
      if (g == 0) {
        to[D] = most[mt] == -INFINITY ? -INFINITY : base[mt];
        to[D + 1] = l[mt];
      }
    }
    __syncthreads();
    for (int e = tid; e < rows_here * (D / 4); e += kThreads) {
      const int r = e / (D / 4), dim = e % (D / 4) * 4;
      const float* at = lds + r * kRowF;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) M = fmaxf(M, at[w * A.lds_rows * kRowF + D]);
      const float base = M == -INFINITY ? 0.0f : M;
      f32x4 sum = {0, 0, 0, 0};
      float L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* aw = at + w * A.lds_rows * kRowF;
        const float f = fast_exp2(0.5f * (aw[D] - base));
        sum += *reinterpret_cast<const f32x4*>(aw + dim) * (f * f);
        L += aw[D + 1] * f * f;
      }
      sum = L == 0.0f ? f32x4{0, 0, 0, 0} : sum * (1.0f / kUnit) * __builtin_amdgcn_rcpf(L) * vtop;
      const size_t row = size_t(n) * A.R + r0 + r;
      if (alone) {
        finish(A, row, D, dim, sum, L, base);
      } else {
        const size_t at_piece = row * A.pieces + piece;
        *reinterpret_cast<f32x4*>(A.part + at_piece * D + dim) = sum;
        if (dim == 0) {
          A.stat[at_piece * 2] = M;
          A.stat[at_piece * 2 + 1] = L;
        }
      }
    }
  }
}

// Joins the pieces of one row, each weighted by its l: D/4 lanes read one
// piece's outputs, the workgroup 1024/D pieces at a time.
template <int D>
__global__ __launch_bounds__(kThreads) void k_q8_join(Args A) {
  constexpr int kLanes = D / 4, kAtOnce = kThreads / kLanes;
  __shared__ __align__(16) float sums[kAtOnce][D];
  const int b = int(quot(A.by_H, A.n0 + quot(A.by_R, blockIdx.x)));
  const size_t row = size_t(A.n0) * A.R + blockIdx.x;
  const int len = q8_len(A.c, b), chunk = q8_chunk(len, A.R);
  if (len <= chunk) return;
  const int pieces = (len + chunk - 1) / chunk, lane = threadIdx.x & 63;
  const int group = threadIdx.x / kLanes, dim = threadIdx.x % kLanes * 4;
  const f32x2* st = reinterpret_cast<const f32x2*>(A.stat) + row * A.pieces;
  const float* part = A.part + row * A.pieces * D + dim;
  f32x2 ml = {-INFINITY, 0.0f};  // the lane's piece of the first 64
  if (lane < pieces) ml = st[lane];
  float M = ml.x;
  for (int p = lane + 64; p < pieces; p += 64) M = fmaxf(M, st[p].x);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off));
  const float base = M == -INFINITY ? 0.0f : M;
  float f = fast_exp2(0.5f * (ml.x - base)), L = ml.y * f * f;
  for (int p = lane + 64; p < pieces; p += 64) {
    f = fast_exp2(0.5f * (st[p].x - base));
    L = __builtin_fmaf(st[p].y * f, f, L);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) L += __shfl_xor(L, off);
  const float by_L = L == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(L);
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
  for (int p = group; p < pieces; p += kAtOnce) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(part + size_t(p) * D);
    const f32x2 w = st[p];
    const float f = fast_exp2(0.5f * (w.x - base));
    sum += x * (w.y * f * f * by_L);
  }
  *reinterpret_cast<f32x4*>(&sums[group][dim]) = sum;
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  f32x4 out = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) out += *reinterpret_cast<const f32x4*>(&sums[i][dim]);
  finish(A, row, D, dim, out, L, base);
}

template <int D, int FMT, int MT, int GROUP, bool STREAM>
void attend(Args A, hipStream_t s) {
  // At most 2^23 workgroups a launch (the grid counts work-items in 32 bits), in
  // whole eights of units.
  const int heads = A.c.B * A.c.H, blocks = (A.R + MT * 16 - 1) / (MT * 16);
  const int room = ((1 << 23) / blocks) & ~7;
  const int most = room / A.pieces > 0 ? room / A.pieces : 1;
  A.by_blocks = fast_div(uint32_t(blocks));
  A.lds_rows = A.R < 16 ? A.R : 16;
  const size_t keys = size_t(q8_longest_chunk(A.c.cap, A.R)) / GROUP * sizeof(Where);
  const size_t sums = size_t(kWaves) * A.lds_rows * (D + 4) * sizeof(float);
  for (A.n0 = 0; A.n0 < heads; A.n0 += most) {
    const int nh = heads - A.n0 < most ? heads - A.n0 : most;
    A.units = nh * A.pieces;
    for (A.unit0 = 0; A.unit0 < A.units; A.unit0 += room) {
      const int here = A.units - A.unit0 < room ? A.units - A.unit0 : room;
      k_q8_attend<D, FMT, MT, GROUP, STREAM>
          <<<unsigned((here + 7) / 8) * 8u * unsigned(blocks), kThreads, keys > sums ? keys : sums,
             s>>>(A);
    }
  }
  if (A.pieces == 1) return;
  const int most_joined = (1 << 23) / A.R;
  for (A.n0 = 0; A.n0 < heads; A.n0 += most_joined) {
    const int nh = heads - A.n0 < most_joined ? heads - A.n0 : most_joined;
    k_q8_join<D><<<unsigned(nh) * unsigned(A.R), kThreads, 0, s>>>(A);
  }
}

template <int D, int FMT>
void attend_rows(const Args& A, hipStream_t s) {
  const bool fours = A.c.bs % 4 == 0;
  // Keys and values that one row block reads, out of pools that are a good part of the
  // last-level cache (256 MB), are read past the caches, which they would only empty.
  // 51 us against 55 on one sequence of 131072 keys (270 MB), 56 against 60 on 512
  // heads of 2048 keys, 30 against 32 on 8 heads of 65536; on pools of 70 MB, found
  // there again by the next call, 22.2 against 20.8.
  const bool stream = uint64_t(A.c.n_blocks) * A.c.H * A.c.bs * D * 2 > (uint64_t(96) << 20);
  // Rows by 16 a workgroup where the last one of 32 would be half empty: 40 rows on
  // 128 heads of 4096 keys take 67 us by 16 and 75 by 32 (D = 64: 40 and 42), 72 rows
  // 99 and 104 (59 and 57), 104 rows 134 and 137 (79 and 72).  An even number of
  // 16s is as fast or faster by 32 (32 rows: 52 and 51).
  const int n = (A.R + 15) / 16;
  if (n % 2 == 1 && n <= (D == 128 ? 7 : 3)) {
    if (fours && stream && n == 1) attend<D, FMT, 1, 4, true>(A, s);
    else if (fours) attend<D, FMT, 1, 4, false>(A, s);
    else attend<D, FMT, 1, 1, false>(A, s);
  } else {
    if (fours) attend<D, FMT, 2, 4, false>(A, s);
    else attend<D, FMT, 2, 1, false>(A, s);
  }
}

}  // namespace

hipError_t launch_q8_attend(const Q8& c, int G, int W, float c_log2, const void* q, void* out,
                            float* lse, float* part, hipStream_t s) {
  Args A;
  A.c = c;
  A.W = W;
  A.R = G * W;
  A.pieces = q8_max_pieces(c.cap, A.R);
  A.n0 = 0;
  A.by_W = fast_div(uint32_t(W));
  A.by_R = fast_div(uint32_t(A.R));
  A.by_pieces = fast_div(uint32_t(A.pieces));
  A.by_H = fast_div(uint32_t(c.H));
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
