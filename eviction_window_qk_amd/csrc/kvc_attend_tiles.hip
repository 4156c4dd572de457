// Causal attention of many rows per KV head on gfx950: packed prompts, and chunks of new
// tokens over a paged cache.
//
// A sequence's n new tokens and the G query heads of a KV head form R = G*n rows (row
// r: token r / G, head r % G).  A workgroup takes 128 rows, 32 a wave, and streams
// their keys and values through LDS in tiles of 64 keys, so that each tile is read
// once for all of them; with many rows the bound is the matrix cores (4*d flops a
// row and key) and, beside them, the vector ALU: one FMA, one exp2, one add and half
// a conversion a score.
//
// Both products are taken transposed, S' = K Q' and O' = V' P', on 32x32x16 matrix
// instructions.  The accumulator gives each lane one query row and 16 of a block's 32
// keys, so the softmax is lane-local, and the weights a lane holds are the ones that
// the second product wants from it: lane half h holds keys 8i + 4h + (0..3), and any
// numbering of the keys serves a product as long as V is read in the same one.  V is
// turned on its way out of LDS (transposing reads of 4 keys x 16 values).
//
// The reference m of a row (w = 2^(x - m)) is not the running maximum: any value serves
// as long as no sum overflows, so a block is summed against the present one and m moves
// to the row's maximum only when a lane's sum passes 2^32 (the first block always
// does).
//
// Tiles go from global memory to LDS without passing registers, one tile ahead, in
// the order in which the LDS banks serve both kinds of reads: 16-byte piece p of row
// r sits at place p ^ swizzle(r).
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kRows = kWaves * 32;   // rows of a workgroup
constexpr int kTile = 64;            // keys of a tile
constexpr int kXcds = 8;
constexpr float kFar = 0x1p64f;      // -m of a row that has seen nothing

struct Args {
  Chunks k;
  int G, H;
  float c_log2;
  Rows q, kr, vr, out;
  float* lse;
  FastDiv by_G;
  int tiles;          // row tiles of the call, counting one spare a sequence
  int parts, per;     // ways a head's row tiles are dealt out to the XCDs, tiles in each
  FastDiv by_per, by_parts;
};

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  return uint32_t(to_bf16(a)) | uint32_t(to_bf16(b)) << 16;
}

// Place of a row's 16-byte pieces: 16 rows' same piece lie in 16 different places of
// the 64 banks (K is read so), and so do four consecutive rows' four neighbouring pieces
// (V).  Two rows of 64 values fill the banks once.
template <int D>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (D == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
  else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}

typedef __attribute__((address_space(3))) void* LdsPtr;

__device__ __forceinline__ void to_lds(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (LdsPtr)to, 16, 0, 0);
}
__device__ __forceinline__ u32x2 read_turned(const uint16_t* at) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
}

// What a row tile works on: its sequence, KV head and rows.
struct Where {
  int b, h, r0, R;   // first row, rows of the sequence
  int token0, n;     // first new token and their count
};

// Row tiles are numbered through: those of sequence b start at floor(starts[b] * G /
// kRows) + b, which leaves room for all of them.  Workgroups go to the XCDs in turn;
// an XCD takes whole parts of heads (all tiles of one head, or every parts-th where
// the heads do not fill the XCDs evenly), the last rows first: they see most keys.
__device__ __forceinline__ bool find(const Args& A, Where& w) {
  const uint32_t x = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
  const uint32_t nth = quot(A.by_per, i);
  const uint32_t unit = nth * kXcds + x;                 // (head, part)
  const uint32_t h = quot(A.by_parts, unit);
  if (h >= uint32_t(A.H)) return false;
  const int tile = A.tiles - 1 - (int(i - nth * A.per) * A.parts + int(unit - h * A.parts));
  if (tile < 0) return false;
  const int G = A.G;
  const auto first = [G](int s, int b) { return int(int64_t(s) * G / kRows) + b; };
  w.b = last_at_or_below(A.k.starts, A.k.B, tile, first);
  const int2 mine = chunk_of(A.k, w.b);
  w.h = int(h);
  w.token0 = mine.x;
  w.n = mine.y;
  w.R = mine.y * G;
  w.r0 = (tile - first(A.k.starts[w.b], w.b)) * kRows;
  return w.r0 >= 0 && w.r0 < w.R;
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void k_prompt(Args A) {
  constexpr int kPieces = D / 8;             // 16-byte pieces of a row
  constexpr int kRowsPerLoad = 64 / kPieces; // rows one wave's load covers
  constexpr int kLoads = kTile / kWaves / kRowsPerLoad;
  constexpr int kSteps = D / 16;             // matrix steps over the head dimension
  constexpr int kDims = D / 32;              // 32-value blocks of the output
  __shared__ __align__(16) uint16_t ks[2][kTile * D];
  __shared__ __align__(16) uint16_t vs[2][kTile * D];

  Where w;
  if (!find(A, w)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 31, hh = lane >> 5;
  const int r = w.r0 + wave * 32 + j;
  const int rc = r < w.R ? r : w.R - 1;      // rows that are none repeat the last one, never written
  const int i = int(quot(A.by_G, uint32_t(rc)));
  const int head = w.h * A.G + rc - i * A.G;
  const int limit = i;                       // last key this row sees
  const int low = __builtin_amdgcn_readfirstlane(limit);
  const int high = __builtin_amdgcn_readlane(limit, 31);
  const int last_row = w.r0 + kRows <= w.R ? w.r0 + kRows - 1 : w.R - 1;
  const int keys = int(quot(A.by_G, uint32_t(last_row))) + 1;   // that any row of the tile sees

  u32x4 qf[kSteps];
  const uint16_t* qp = A.q.p + int64_t(w.token0 + i) * A.q.ts + int64_t(head) * A.q.hs + hh * 8;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + s * 16);

  const uint16_t* kb = A.kr.p + int64_t(w.token0) * A.kr.ts + int64_t(w.h) * A.kr.hs;
  const uint16_t* vb = A.vr.p + int64_t(w.token0) * A.vr.ts + int64_t(w.h) * A.vr.hs;
  // Rows past the sequence's end repeat its last one: they are in bounds, and no row
  // sees them.
  auto fetch = [&](int t0, int buf) {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int first = wave * (kTile / kWaves) + x * kRowsPerLoad, row = first + lane / kPieces;
      const int t = t0 + row < w.n ? t0 + row : w.n - 1;
      const int piece = (lane % kPieces) ^ swizzle<D>(row);
      to_lds(kb + int64_t(t) * A.kr.ts + piece * 8, ks[buf] + first * D);
      to_lds(vb + int64_t(t) * A.vr.ts + piece * 8, vs[buf] + first * D);
    }
  };

  f32x16 acc[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d) acc[d] = f32x16{};
  float nm = kFar, l = 0.0f;
  const float by = A.c_log2;

  fetch(0, 0);
  const int n_tiles = (keys + kTile - 1) / kTile;
  for (int tile = 0; tile < n_tiles; ++tile) {
    const int t0 = tile * kTile;
    __builtin_amdgcn_s_waitcnt(0);           // this tile's loads, one tile old
    __syncthreads();
    if (tile + 1 < n_tiles) fetch(t0 + kTile, (tile + 1) & 1);
    if (t0 > high) continue;                 // no row of this wave sees it
    const uint16_t* kt = ks[tile & 1];
    const uint16_t* vt = vs[tile & 1];
    f32x16 sc[2];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      sc[blk] = f32x16{};
      const int row = blk * 32 + j;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int place = (2 * s + hh) ^ swizzle<D>(row);
        sc[blk] = mfma(*reinterpret_cast<const u32x4*>(kt + row * D + place * 8), qf[s], sc[blk]);
      }
    }
    if (t0 + kTile - 1 > low) {
      const int d = limit - t0 - 4 * hh;
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (blk * 32 + 8 * (e >> 2) + (e & 3) > d) sc[blk][e] = -INFINITY;
    }
    float p[32], sum = 0.0f;
    auto weigh = [&]() {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        p[e] = fast_exp2(__builtin_fmaf(sc[e >> 4][e & 15], by, nm));
        p[e + 1] = fast_exp2(__builtin_fmaf(sc[e >> 4][(e & 15) + 1], by, nm));
        s0 += p[e];
        s1 += p[e + 1];
      }
      sum = s0 + s1;
    };
    weigh();
    if (__any(!(sum <= 0x1p32f))) {
      float top = sc[0][0];
#pragma unroll
      for (int e = 1; e < 32; ++e) top = fmaxf(top, sc[e >> 4][e & 15]);
      top = fmaxf(top, __shfl_xor(top, 32));
      const float now = fminf(nm, -top * by), f = fast_exp2(now - nm);
      nm = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] *= f;
      weigh();
    }
    l += sum;
#pragma unroll
    for (int s = 0; s < 4; ++s) {            // 16 keys a step
      const u32x4 pf = {pack(p[8 * s], p[8 * s + 1]), pack(p[8 * s + 2], p[8 * s + 3]),
                        pack(p[8 * s + 4], p[8 * s + 5]), pack(p[8 * s + 6], p[8 * s + 7])};
#pragma unroll
      for (int d = 0; d < kDims; ++d) {
        // lane: 4 keys from 16s + 4hh (and 8 further on), values 32d + 16 ((lane >> 4) & 1) +
        // 4 (lane & 3).., of which it gets the four keys of value 32d + j
        const int row = 16 * s + 4 * hh + ((lane & 15) >> 2);
        const int col = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        const int at0 = row * D + (((col >> 3) ^ swizzle<D>(row)) << 3) + (col & 7);
        const int at1 = (row + 8) * D + (((col >> 3) ^ swizzle<D>(row + 8)) << 3) + (col & 7);
        const u32x2 a = read_turned(vt + at0), b = read_turned(vt + at1);
        acc[d] = mfma(u32x4{a.x, a.y, b.x, b.y}, pf, acc[d]);
      }
    }
  }

  l += __shfl_xor(l, 32);
  if (r >= w.R) return;
  const bool any = l > 0.0f;
  const float by_l = any ? 1.0f / l : 0.0f;
  uint16_t* to = A.out.p + int64_t(w.token0 + i) * A.out.ts + int64_t(head) * A.out.hs;
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u16x4*>(to + 32 * d + 8 * e + 4 * hh) =
          u16x4{to_bf16(acc[d][4 * e] * by_l), to_bf16(acc[d][4 * e + 1] * by_l),
                to_bf16(acc[d][4 * e + 2] * by_l), to_bf16(acc[d][4 * e + 3] * by_l)};
  if (A.lse && hh == 0)
    A.lse[size_t(w.token0 + i) * (A.G * A.H) + head] =
        any ? (fast_log2(l) - nm) * 0.6931471805599453f : -INFINITY;
}

// Row tiles, and how the heads' are dealt out to the XCDs.
void deal(Args& A) {
  A.tiles = int(int64_t(A.k.n_tokens) * A.G / kRows) + A.k.B;
  A.parts = kXcds;
  for (int h = A.H; h % 2 == 0 && A.parts > 1; h /= 2) A.parts /= 2;
  A.per = (A.tiles + A.parts - 1) / A.parts;
  A.by_per = fast_div(uint32_t(A.per));
  A.by_parts = fast_div(uint32_t(A.parts));
  A.by_G = fast_div(uint32_t(A.G));
}

}  // namespace

hipError_t launch_prompt_attend(int H, int G, int D, const Chunks& k, float c_log2, const Rows& q,
                                const Rows& k_rows, const Rows& v_rows, const Rows& out,
                                float* lse, hipStream_t s) {
  Args A{};
  A.k = k;
  A.G = G;
  A.H = H;
  A.c_log2 = c_log2;
  A.q = q, A.kr = k_rows, A.vr = v_rows, A.out = out;
  A.lse = lse;
  deal(A);
  const unsigned blocks = unsigned((int64_t(H) * A.parts + kXcds - 1) / kXcds * kXcds * A.per);
  if (D == 128) k_prompt<128><<<blocks, kThreads, 0, s>>>(A);
  else k_prompt<64><<<blocks, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kvc
