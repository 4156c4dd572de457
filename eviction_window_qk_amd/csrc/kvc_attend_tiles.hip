// Causal attention of many rows per KV head on gfx950: packed prompts, and chunks of new
// tokens over a paged cache.
//
// A sequence's n new tokens and the G query heads of a KV head form R = G*n rows (row
// r: token r / G, head r % G).  A workgroup takes 128 or 256 rows, 32 a wave, and streams
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
// does).  Values so large that their sums pass fp32 before that are taken a second
// time, with smaller weights (loud_of).
//
// Tiles go from global memory to LDS without passing registers, one tile ahead, in
// the order in which the LDS banks serve both kinds of reads: 16-byte piece p of row
// r sits at place p ^ swizzle(r).  Eight waves share a CU, so that one's softmax runs
// beside another's products.
//
// Measured, machine to machine: a 16384-token prompt, 8 KV heads of 128, 4 rows a token,
// 1910 to 2000 us (1150 to 1100 TFLOP/s, matrix cores busy 53 % at 1.9 GHz; a library product of
// 8192^3 reaches 1232 to 1268); of 64 values 1105 to 1210 us (995 to 909).  512 tokens over 131072
// slots 970 to 1060 us (1130 to 1040).  With four waves a workgroup the prompt took 2025 us
// where it takes 1970 with eight, and in copies of the kernel 1761 without the loads to
// LDS, 1961 without exp2, 1971 with half of the reads of V.
#include <type_traits>

#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kRows = kTileRows;     // rows of a workgroup, 32 a wave
constexpr int kTile = 64;            // keys of a tile
constexpr int kXcds = 8;
constexpr float kFar = 0x1p64f;      // -m of a row that has seen nothing
static_assert(kRows == kWaves * 32, "32 rows a wave");

struct Args {
  Paged c;            // of a call over a cache
  Chunks k;
  int G, H;
  float c_log2;
  Rows q, kr, vr, out;  // kr, vr: keys and values of a call without a cache
  float* lse;
  FastDiv by_G;
  int slots;          // workgroups of a head
  int parts, per;     // ways a head's slots are dealt out to the XCDs, slots in each
  FastDiv by_per, by_parts;
  int most;           // pieces that any sequence is cut into
  Partials places;    // of a sequence [piece][row], outputs [piece][D / 4][row][4]
};

// Rows past the end, or in no page, are read from here.
__device__ const u32x4 zeros[16] = {};

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Place of a row's 16-byte pieces: 16 rows' same piece lie in 16 different places of
// the 64 banks (K is read so), and so do four consecutive rows' four neighbouring pieces
// (V).  Two rows of 64 values fill the banks once.
template <int D>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (D == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
  else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}

// 16 bytes a lane from global memory to LDS, lane l's to `to` + 16 l, past the registers.
// In assembly, as the compiler takes the builtin's store for one that any later read of
// LDS may want, and waits for the tile on its way before it reads the one that is there
// (512 tokens over 131072 slots 1220 us for 1147, a 16384-token prompt 2056 for 2025).
// m0 is a register that the compiler reserves (it warns where it is named as clobbered): it
// keeps nothing there, and these kernels have no other instruction that reads it.
// The instruction writes no register; whoever reads the tile waits for it (s_waitcnt) and
// meets the other waves (barrier) first.
__device__ __forceinline__ void to_lds(const void* from, const void* to) {
  const uint32_t at = uint32_t(uintptr_t((__attribute__((address_space(3))) const void*)to));
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(from), "s"(__builtin_amdgcn_readfirstlane(at)) : "memory");
}
__device__ __forceinline__ u32x2 read_turned(const uint16_t* at) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
}

// What a workgroup works on: its sequence, KV head, rows and piece of the keys.
struct Where {
  int b, h, first;    // first: of the sequence's slots
  int r0, R;          // first row, rows of the sequence
  int token0, n;      // first new token and their count
  int len;            // keys of the sequence
  int piece, pieces, tiles;
};

// A head's work is numbered through in slots, (piece, row tile) pairs: those of
// sequence b start at first_slot, which leaves room for all of them.  Workgroups go to
// the XCDs in turn; an XCD takes whole parts of heads (all slots of one head, or every
// parts-th where the heads do not fill the XCDs evenly), the last rows first: they see
// most keys.  The row tiles of a piece follow each other on one XCD, whose L2 then reads
// the keys once.
template <bool PAGED, int kW>
__device__ __forceinline__ bool find(const Args& A, Where& w) {
  constexpr int kHere = kW * 32;                         // rows of a workgroup
  const uint32_t x = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
  const uint32_t nth = quot(A.by_per, i);
  const uint32_t unit = nth * kXcds + x;                 // (head, part)
  const uint32_t h = quot(A.by_parts, unit);
  if (h >= uint32_t(A.H)) return false;
  const int at = int(i - nth * A.per) * A.parts + int(unit - h * A.parts);
  const int slot = A.slots - 1 - at;
  if (slot < 0) return false;
  const int G = A.G, most = A.most;
  const auto first = [G, most](int s, int b) { return PAGED ? first_slot(s, b, G, most) : first_tile(s, b, G, kHere); };
  w.b = last_at_or_below(A.k, slot, first);
  const int2 mine = chunk_of(A.k, w.b);
  w.h = int(h);
  w.token0 = mine.x;
  w.n = mine.y;
  w.R = mine.y * G;
  w.first = first(mine.x, w.b);
  const int s = slot - w.first;
  w.tiles = (w.R + kRows - 1) / kRows;
  if (PAGED) {
    if (w.R <= kFewRows || s < 0) return false;
    w.len = paged_len(A.c, w.b);
    w.pieces = tile_pieces(w.len, w.tiles);
    const int here = (w.R + kHere - 1) / kHere;
    w.piece = s / here;
    if (w.piece >= w.pieces || w.first + w.tiles * w.pieces > A.slots) return false;
    w.r0 = (s - w.piece * here) * kHere;
    return true;
  }
  w.len = w.n;
  w.piece = 0;
  w.pieces = 1;
  w.r0 = s * kHere;
  return s >= 0 && w.r0 < w.R;
}

// What a workgroup computes, with threads counted by `thread`.  Returns whether any wave's results
// are not finite; such waves leave their results to a second call (LOUD), in which the others help to
// load.  A wave decides for itself: its rows are the same whatever kW.
// kW: waves of a workgroup.  GROUP: keys that a look-up in the table covers, of a wave's load all where pages hold
// whole loads, or one; 0: no cache.
template <int D, int GROUP, int kW, bool LOUD>
__device__ __forceinline__ bool attend_tiles(const Args& A, int thread, bool& wanted, uint16_t (&ks)[2][kTile * D],
                                             uint16_t (&vs)[2][kTile * D], int (&flags)[kW]) {
  constexpr bool PAGED = GROUP != 0;
  constexpr int kPieces = D / 8;             // 16-byte pieces of a row
  constexpr int kRowsPerLoad = 64 / kPieces; // rows one wave's load covers
  constexpr int kLoads = kTile / kW / kRowsPerLoad;
  constexpr int kSteps = D / 16;             // matrix steps over the head dimension
  constexpr int kDims = D / 32;              // 32-value blocks of the output
  constexpr int kPerTile = PAGED ? kTile / GROUP : 1;    // look-ups of a tile
  constexpr int kBatch = PAGED ? 64 / kPerTile : 1;      // tiles that a wave's 64 look-ups cover
  static_assert(GROUP == 0 || GROUP == 1 || GROUP == kRowsPerLoad, "a load's rows, or one");

  Where w;
  if (!find<PAGED, kW>(A, w)) return false;
  const int lane = thread & 63;
  const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
  const int j = lane & 31, hh = lane >> 5;
  const int r = w.r0 + wave * 32 + j;
  const int rc = r < w.R ? r : w.R - 1;      // rows that are none repeat the last one, never written
  const int i = int(quot(A.by_G, uint32_t(rc)));
  const int head = w.h * A.G + rc - i * A.G;
  const int limit = w.len - w.n + i;         // last key this row sees
  const int low = __builtin_amdgcn_readfirstlane(limit);
  // A wave without rows helps to load.
  const int high = w.r0 + wave * 32 < w.R ? __builtin_amdgcn_readlane(limit, 31) : -1;
  const int last_row = w.r0 + kW * 32 <= w.R ? w.r0 + kW * 32 - 1 : w.R - 1;
  // Keys that any row of the tile sees, of these the piece's.
  const int seen = w.len - w.n + int(quot(A.by_G, uint32_t(last_row))) + 1;
  const int span = PAGED ? tile_span(w.len, w.pieces) : 0;
  const int from = w.piece * span;
  const int to = PAGED && from + span < seen ? from + span : seen;

  u32x4 qf[kSteps];
  const uint16_t* qp = A.q.p + int64_t(w.token0 + i) * A.q.ts + int64_t(head) * A.q.hs + hh * 8;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + s * 16);

  // Where the keys are.  Without a cache, rows past the sequence's end repeat its last
  // one: they are in bounds, and no row sees them.  In a cache a wave's 64 lanes look up
  // kBatch tiles at a time, one batch ahead: the row in the pools, or kNone.
  constexpr uint32_t kNone = 0xffffffffu;
  const uint16_t* kb = A.kr.p + int64_t(w.token0) * A.kr.ts + int64_t(w.h) * A.kr.hs;
  const uint16_t* vb = A.vr.p + int64_t(w.token0) * A.vr.ts + int64_t(w.h) * A.vr.hs;
  uint32_t rows = kNone, rows_next = kNone;
  auto look_up = [&](int t) {                // of the batch that starts at key t
    const int key = t + lane * (PAGED ? GROUP : 1);
    if (key >= w.len) return kNone;
    const int64_t at = paged_row(A.c, w.b, w.h, key);
    return at < 0 ? kNone : uint32_t(at);
  };
  // Bytes of a lane's piece from its tile's (no cache) or its group's first row: below
  // 2^32, so a load's address is a scalar base and these, added in 64 bits for each load.
  uint32_t k_off[kLoads], v_off[kLoads];
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int row = wave * (kTile / kW) + x * kRowsPerLoad + lane / kPieces;
    const int piece = (lane % kPieces) ^ swizzle<D>(row);
    k_off[x] = PAGED ? uint32_t((lane / kPieces) * D + piece * 8) * 2 : (uint32_t(row) * uint32_t(A.kr.ts) + piece * 8) * 2;
    v_off[x] = PAGED ? k_off[x] : (uint32_t(row) * uint32_t(A.vr.ts) + piece * 8) * 2;
  }
  auto at_off = [](const uint16_t* p, uint32_t off) { return reinterpret_cast<const char*>(p) + off; };
  auto fetch = [&](int t0, int nth, uint32_t of, int buf) {   // nth: tile of the batch
    if constexpr (!PAGED) {
      if (t0 + kTile <= w.n) {
        const uint16_t* kp = kb + int64_t(t0) * A.kr.ts;
        const uint16_t* vp = vb + int64_t(t0) * A.vr.ts;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          const int first = wave * (kTile / kW) + x * kRowsPerLoad;
          to_lds(at_off(kp, k_off[x]), ks[buf] + first * D);
          to_lds(at_off(vp, v_off[x]), vs[buf] + first * D);
        }
        return;
      }
    }
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int first = wave * (kTile / kW) + x * kRowsPerLoad, row = first + lane / kPieces;
      const int piece = (lane % kPieces) ^ swizzle<D>(row);
      if constexpr (!PAGED) {
        const int t = t0 + row < w.n ? t0 + row : w.n - 1;
        to_lds(kb + int64_t(t) * A.kr.ts + piece * 8, ks[buf] + first * D);
        to_lds(vb + int64_t(t) * A.vr.ts + piece * 8, vs[buf] + first * D);
      } else if constexpr (GROUP > 1) {
        const uint32_t at = __builtin_amdgcn_readlane(of, nth * kPerTile + first / GROUP);
        if (at != kNone && t0 + first + GROUP <= w.len) {
          to_lds(at_off(A.c.k + size_t(at) * D, k_off[x]), ks[buf] + first * D);
          to_lds(at_off(A.c.v + size_t(at) * D, k_off[x]), vs[buf] + first * D);
        } else {   // rows past the end may hold anything, and nothing times a NaN is one
          const uint16_t* z = reinterpret_cast<const uint16_t*>(zeros);
          const size_t inner = size_t(at) * D + (lane / kPieces) * D;
          const bool in = at != kNone && t0 + row < w.len;
          to_lds((in ? A.c.k + inner : z) + piece * 8, ks[buf] + first * D);
          to_lds((in ? A.c.v + inner : z) + piece * 8, vs[buf] + first * D);
        }
      } else {
        const uint32_t at = uint32_t(__shfl(int(of), row));
        const uint16_t* kp = at == kNone ? reinterpret_cast<const uint16_t*>(zeros) : A.c.k + size_t(at) * D;
        const uint16_t* vp = at == kNone ? reinterpret_cast<const uint16_t*>(zeros) : A.c.v + size_t(at) * D;
        to_lds(kp + piece * 8, ks[buf] + first * D);
        to_lds(vp + piece * 8, vs[buf] + first * D);
      }
    }
  };

  f32x16 acc[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d) acc[d] = f32x16{};
  float nm = kFar, l = 0.0f;
  const float by = A.c_log2;

  const int n_tiles = to > from ? (to - from + kTile - 1) / kTile : 0;
  // Two lanes a row and tile, of the tiles that the wave's own rows see.
  const int to_here = high + 1 < to ? high + 1 : to;
  const Loud loud = LOUD ? loud_of(to_here > from ? 2 * ((to_here - from + kTile - 1) / kTile) : 1) : Loud{kSumLimit, 0.0f};
  if (PAGED) rows = look_up(from);
  if (n_tiles > 0) fetch(from, 0, rows, 0);
  if (PAGED && n_tiles > kBatch) rows_next = look_up(from + kBatch * kTile);
  uint64_t none = 0;                         // look-ups of the batch in work that found nothing
  for (int tile = 0; tile < n_tiles; ++tile) {
    const int t0 = from + tile * kTile;
    uint32_t gone = 0;                       // GROUP > 1: those of this tile
    uint64_t gone1 = 0;                      // GROUP 1
    if constexpr (PAGED) {
      const int nth = tile % kBatch;
      if (nth == 0) none = __ballot(rows == kNone);
      if constexpr (GROUP > 1) gone = uint32_t(none >> (nth * kPerTile)) & ((1u << kPerTile) - 1);
      else gone1 = none;
    }
    __builtin_amdgcn_s_waitcnt(0);           // this tile's loads, one tile old
    __syncthreads();
    if (tile + 1 < n_tiles) {
      const int nth = (tile + 1) % kBatch;
      if (PAGED && nth == 0) {
        rows = rows_next;
        if (tile + 1 + kBatch < n_tiles) rows_next = look_up(t0 + kTile + kBatch * kTile);
      }
      fetch(t0 + kTile, nth, rows, (tile + 1) & 1);
    }
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
    if (t0 + kTile - 1 > low || gone != 0 || gone1 != 0) {
      int d = limit - t0 - 4 * hh;
      asm volatile("" : "+v"(d));            // a branch: not 32 selects in every tile
      // bit k / GROUP: key k + 4 hh of the tile
      const uint32_t g_lane = GROUP == 4 ? gone >> hh : gone;
      const uint64_t g_one = gone1 >> (4 * hh);
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = blk * 32 + 8 * (e >> 2) + (e & 3);
          bool out = k > d;
          if constexpr (GROUP > 1) out |= (g_lane >> (k / GROUP)) & 1;
          if constexpr (GROUP == 1) out |= (g_one >> k) & 1;
          if (out) sc[blk][e] = -INFINITY;
        }
    }
    // Matrix instructions go first where the SIMD's two waves want to issue: the one in its
    // softmax fills the gaps (16384-token prompt -1.5 %, 512 tokens over 131072 slots
    // -4.5 %; the softmax first: +3.6 %, -1 %).
    __builtin_amdgcn_s_setprio(0);
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
    if (__any(!(sum <= loud.limit))) {
      float top = sc[0][0];
#pragma unroll
      for (int e = 1; e < 32; ++e) top = fmaxf(top, sc[e >> 4][e & 15]);
      top = fmaxf(top, __shfl_xor(top, 32));
      const float now = fminf(nm, -top * by - loud.lift), f = fast_exp2(now - nm);
      nm = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] *= f;
      weigh();
    }
    l += sum;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {            // 16 keys a step
      const u32x4 pf = {pack_bf16(p[8 * s], p[8 * s + 1]), pack_bf16(p[8 * s + 2], p[8 * s + 3]),
                        pack_bf16(p[8 * s + 4], p[8 * s + 5]), pack_bf16(p[8 * s + 6], p[8 * s + 7])};
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
  const bool any = l > 0.0f;
  const float by_l = any ? 1.0f / l : 0.0f;
  const float b_sum = any ? fast_log2(l) - nm : -INFINITY;   // log2 of the row's sum of 2^x
  u32x2 out[kDims][4];
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      acc[d][e] *= by_l;
      if constexpr (LOUD) acc[d][e] = within_bf16(acc[d][e]);
    }
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      out[d][e] = u32x2{pack_bf16(acc[d][4 * e], acc[d][4 * e + 1]), pack_bf16(acc[d][4 * e + 2], acc[d][4 * e + 3])};
  bool more = false;
  if constexpr (!LOUD) {
    // Nothing times infinity or NaN is NaN: a row's two lanes at once, beside the vector ALU, which
    // would take 64 steps (eleven prompts of 2043 tokens on average +3 %).
    f32x16 none_of = {};
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        none_of = mfma(u32x4{0, 0, 0, 0}, u32x4{out[d][e].x, out[d][e].y, out[d][e + 1].x, out[d][e + 1].y}, none_of);
    wanted = __any(none_of[0] != none_of[0]);
    if (lane == 0) flags[wave] = wanted;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kW; ++x) more |= flags[x] != 0;
  }
  if (r >= w.R || wanted != LOUD) return more;
  if (PAGED && w.pieces > 1) {
    const size_t at = size_t(w.h) * A.places.total + first_place(A.places, w.token0, w.b, A.G) + w.piece * w.R;
    float* po = A.places.part + at * D + r * 4;
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(po + size_t(32 * d + 8 * e + 4 * hh) * w.R) =
            f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]};
    if (hh == 0) A.places.stat[at + r] = b_sum;
    return more;
  }
  uint16_t* po = A.out.p + int64_t(w.token0 + i) * A.out.ts + int64_t(head) * A.out.hs;
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<u32x2*>(po + 32 * d + 8 * e + 4 * hh) = out[d][e];
  if (A.lse && hh == 0)
    A.lse[size_t(w.token0 + i) * (A.G * A.H) + head] = b_sum * 0.6931471805599453f;
  return more;
}

template <int D, int GROUP, int kW>
__global__ __launch_bounds__(kW * 64, 2) void k_attend_tiles(Args A) {
  __shared__ __align__(16) uint16_t ks[2][kTile * D];
  __shared__ __align__(16) uint16_t vs[2][kTile * D];
  __shared__ int flags[kW];
  bool wanted = false;
  int thread = threadIdx.x;
  if (attend_tiles<D, GROUP, kW, false>(A, thread, wanted, ks, vs, flags)) {
    asm volatile("" : "+v"(thread));         // or what the two calls share stays in registers
    attend_tiles<D, GROUP, kW, true>(A, thread, wanted, ks, vs, flags);
  }
}

// Joins the pieces of 1024 / D rows of a row tile, each weighted by its sum, four values
// a lane, in the partials' order: 4 D bytes a row and piece, 15 us of the 270 of a mixed
// batch (24 sequences of up to 16384 slots of 8 heads of 64, 1183 new tokens).
template <int D>
__global__ __launch_bounds__(kThreads) void k_join_tiles(Args A, FastDiv by_tiles) {
  constexpr int kLanes = D / 4, kAtOnce = kThreads / kLanes;
  const int G = A.G;
  const int h = int(quot(by_tiles, blockIdx.x)), tile = int(blockIdx.x) - h * int(by_tiles.d);
  const int b = last_at_or_below(A.k, tile, [G](int s, int i) { return first_tile(s, i, G); });
  const int2 mine = chunk_of(A.k, b);
  const int R = mine.y * G, start = mine.x, t = tile - first_tile(start, b, G);
  if (R <= kFewRows || t < 0) return;
  const int tiles = (R + kRows - 1) / kRows, pieces = tile_pieces(paged_len(A.c, b), tiles);
  const int in_tile = int(blockIdx.y) * kAtOnce + int(threadIdx.x) % kAtOnce, r = t * kRows + in_tile;
  if (pieces == 1 || r >= R) return;
  const int dim = threadIdx.x / kAtOnce * 4;
  const size_t at = size_t(h) * A.places.total + first_place(A.places, start, b, G);
  const float* part = A.places.part + at * D + (size_t(dim) * R + r * 4);
  const float* stat = A.places.stat + at + r;
  const size_t step = R;                                 // from piece to piece
  float M = -INFINITY;
#pragma unroll 4
  for (int p = 0; p < pieces; ++p) M = fmaxf(M, stat[p * step]);
  const float base = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
  for (int p = 0; p < pieces; ++p) {
    const float f = fast_exp2(stat[p * step] - base);
    sum += *reinterpret_cast<const f32x4*>(part + p * step * D) * f;
    L += f;
  }
  const float by_l = L > 0.0f ? 1.0f / L : 0.0f;
  if (unless_finite(sum.x, sum.y, sum.z, sum.w) == 0.0f) {
    sum *= by_l;
  } else {                                               // each piece's share first
    sum = f32x4{0, 0, 0, 0};
    for (int p = 0; p < pieces; ++p)
      sum += *reinterpret_cast<const f32x4*>(part + p * step * D) * (fast_exp2(stat[p * step] - base) * by_l);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) sum[x] = within_bf16(sum[x]);
  const int i = int(quot(A.by_G, uint32_t(r))), head = h * G + r - i * G;
  *reinterpret_cast<u32x2*>(A.out.p + int64_t(mine.x + i) * A.out.ts + int64_t(head) * A.out.hs + dim) =
      u32x2{pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w)};
  if (A.lse && dim == 0)
    A.lse[size_t(mine.x + i) * (G * A.H) + head] =
        L > 0.0f ? (base + fast_log2(L)) * 0.6931471805599453f : -INFINITY;
}

// Column sums of the softmax weights of sequences with many rows: keys stationary, 32 kX a
// wave as the second operand of S = Q K', query rows streamed through LDS 64 at a time.
// The accumulator gives a lane one key and 16 rows, so the sum down the rows is
// lane-local; its order is fixed: every fourth tile of rows makes a sum, and the four are
// added.  kParts 4: by four waves each.  It takes the scores again (2 d flops a row and key): kept,
// they would be 4 bytes of each.  67 us in the mixed batch, bound by exp2 and its FMA and
// add (16 cycles a score for the products' 8) and by the start of short runs of rows.
constexpr int kRuns = 4;
template <int D, int kX, int kParts>
__global__ __launch_bounds__(kParts * kThreads, kParts == 1 ? 2 : 1) void k_weights_tiles(Args A, FastDiv by_chunks, int n0) {
  constexpr int kPieces = D / 8;
  constexpr int kRowsPerLoad = 64 / kPieces;
  constexpr int kLoads = kTile / kWaves / kRowsPerLoad;
  constexpr int kSteps = D / 16;
  static_assert(kParts == 1 || kParts == kRuns, "a part takes all runs, or one");
  __shared__ __align__(16) uint16_t qs_all[kParts][2][kTile * D];
  __shared__ __align__(16) float bs_all[kParts][2][kTile];   // -log2 of the rows' sums
  __shared__ __align__(16) int lim_all[kParts][2][kTile];    // the rows' last keys
  const int part = kParts == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads), tid = threadIdx.x % kThreads;
  auto& qs = qs_all[part];
  auto& bs = bs_all[part];
  auto& lim = lim_all[part];
  const int nth = int(quot(by_chunks, blockIdx.x)), n = n0 + nth, b = n / A.H, h = n - b * A.H;
  const int2 mine = chunk_of(A.k, b);
  const int R = mine.y * A.G, len = paged_len(A.c, b);
  if (R <= kFewRows) return;
  const int t0 = (int(blockIdx.x) - nth * int(by_chunks.d)) * (kWaves * 32 * kX);
  if (t0 >= len) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane & 31, hh = lane >> 5;
  const int key0 = t0 + wave * 32 * kX;
  u32x4 kf[kX][kSteps];
  bool there[kX];
#pragma unroll
  for (int x = 0; x < kX; ++x) {
    const int t = key0 + x * 32 + j;
    const int64_t row = t < len ? paged_row(A.c, b, h, t) : -1;
    there[x] = row >= 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      kf[x][s] = there[x] ? *reinterpret_cast<const u32x4*>(A.c.k + row * D + s * 16 + hh * 8) : u32x4{0, 0, 0, 0};
  }
  // Rows that see any of the keys: from the first token whose slot is at or past t0, or
  // a 256-key boundary before it, so that a key's rows are added in one order whatever kX.
  const int first_new = len - mine.y, seen_from = t0 & ~255;
  const int tok = seen_from > first_new ? seen_from - first_new : 0;
  const int r_from = tok * A.G, n_tiles = (R - r_from + kTile - 1) / kTile;
  auto fetch = [&](int tile, int buf) {
    const int r0 = r_from + tile * kTile;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int first = wave * (kTile / kWaves) + x * kRowsPerLoad, row = first + lane / kPieces;
      const int r = r0 + row < R ? r0 + row : R - 1, i = int(quot(A.by_G, uint32_t(r)));
      const int piece = (lane % kPieces) ^ swizzle<D>(row);
      to_lds(A.q.p + int64_t(mine.x + i) * A.q.ts + int64_t(h * A.G + r - i * A.G) * A.q.hs + piece * 8, qs[buf] + first * D);
    }
    if (tid < kTile) {
      const int r = r0 + tid, rc = r < R ? r : R - 1, i = int(quot(A.by_G, uint32_t(rc)));
      const float z = A.lse[size_t(mine.x + i) * (A.G * A.H) + h * A.G + rc - i * A.G];
      const bool any = r < R && z != -INFINITY;
      bs[buf][tid] = any ? -z * 1.4426950408889634f : -INFINITY;   // a row that sees nothing gives nothing
      lim[buf][tid] = first_new + i;
    }
  };
  if (part < n_tiles) fetch(part, 0);
  float total[kX] = {}, sum[kX] = {};
  const float by = A.c_log2;
  const int steps = kParts == 1 ? n_tiles : (n_tiles + kRuns - 1) / kRuns;
  int tile = part;
  for (int step = 0; step < steps; ++step) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    const bool last = tile + kRuns >= n_tiles;                     // of its run
    const int next = kParts == 1 && last ? tile % kRuns + 1 : tile + kRuns;
    if (step + 1 < steps && next < n_tiles) fetch(next, (step + 1) & 1);
    if (kParts > 1 && tile >= n_tiles) continue;
    const uint16_t* qt = qs[step & 1];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      f32x16 sc[kX] = {};
      const int row = blk * 32 + j;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const u32x4 qf = *reinterpret_cast<const u32x4*>(qt + row * D + (((2 * s + hh) ^ swizzle<D>(row)) << 3));
#pragma unroll
        for (int x = 0; x < kX; ++x) sc[x] = mfma(qf, kf[x][s], sc[x]);
      }
      auto add = [&](auto checked) {
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const int at = blk * 32 + 8 * e4 + 4 * hh;
          const f32x4 bz = *reinterpret_cast<const f32x4*>(&bs[step & 1][at]);
          i32x4 lm = {0, 0, 0, 0};
          if constexpr (checked) lm = *reinterpret_cast<const i32x4*>(&lim[step & 1][at]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int x = 0; x < kX; ++x) {
              const float p = fast_exp2(__builtin_fmaf(sc[x][4 * e4 + e], by, bz[e]));
              total[x] += !checked || key0 + x * 32 + j <= lm[e] ? p : 0.0f;
            }
        }
      };
      // the tile's first row sees least
      if (key0 + 32 * kX - 1 <= first_new + int(quot(A.by_G, uint32_t(r_from + tile * kTile)))) add(std::false_type{});
      else add(std::true_type{});
    }
    if (kParts == 1 && last) {
#pragma unroll
      for (int x = 0; x < kX; ++x) sum[x] += total[x], total[x] = 0.0f;
    }
    tile = next;
  }
  if constexpr (kParts > 1) {
    float* const sums = reinterpret_cast<float*>(qs_all);   // [part][x][thread]
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kX; ++x) sums[(part * kX + x) * kThreads + tid] = total[x];
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int x = 0; x < kX; ++x)
#pragma unroll
      for (int i = 0; i < kParts; ++i) sum[x] += sums[(i * kX + x) * kThreads + tid];
  }
#pragma unroll
  for (int x = 0; x < kX; ++x) {
    sum[x] += __shfl_xor(sum[x], 32);
    if (hh == 0 && there[x]) A.c.weight[size_t(n) * A.c.room + key0 + x * 32 + j] += sum[x];
  }
}

// How the heads' slots are dealt out to the XCDs.  Returns the workgroups.
unsigned deal(Args& A, int slots) {
  A.slots = slots;
  A.parts = kXcds;
  for (int h = A.H; h % 2 == 0 && A.parts > 1; h /= 2) A.parts /= 2;
  A.per = (slots + A.parts - 1) / A.parts;
  A.by_per = fast_div(uint32_t(A.per));
  A.by_parts = fast_div(uint32_t(A.parts));
  A.by_G = fast_div(uint32_t(A.G));
  return unsigned((int64_t(A.H) * A.parts + kXcds - 1) / kXcds * kXcds * A.per);
}

// Whether workgroups take 256 rows, eight waves, and so half as many loads of keys for their
// products (the results are the same bits: a wave's rows are the same ones).  It pays
// for 128 values (64 are bound by the softmax: 1357 us against 1296 on a 16384-token
// prompt) where they still fill the chip, waste few rows and run long.  Of prompts (us, eight waves :
// four; 8 KV heads, 4 rows a token unless said): 16384 tokens 2224 : 2330, 4096 155 : 161, 11 of 2043 on
// average, 4 heads of 7 rows, 561 : 578, 8 of 2048 342 : 344, 16 of 1024 222 : 209, one of 2048 62 : 57,
// 16384 tokens of one KV head (256 workgroups) 409 : 392.
bool eight_waves(int64_t rows, int seqs, int H, int D) {
  return D == 128 && rows / seqs >= 8192 && rows * H / (2 * kRows) >= 512;
}
// Of chunks over a cache, by the rows of a sequence on average and the longest length: 512 tokens over
// 131072 slots 1149 : 1263, over 16384 162 : 175, over 8192 (pieces of 2048 keys) 91 : 97; 8 of 256
// over 4096 (of 512) 257 : 242, 8 of 64 over 32768 (of 1024) 443 : 431; 512 over 32768 slots of four
// heads (128 workgroups) 226 : 200.
bool eight_waves(const Args& A, int D) {
  const int64_t rows = int64_t(A.k.n_tokens) * A.G / A.k.B;
  if (D != 128 || rows <= kRows) return false;
  const int tiles = int((rows + kRows - 1) / kRows), pieces = tile_pieces(A.c.cap, tiles);
  return tile_span(A.c.cap, pieces) >= 2048 && A.H * int64_t(A.k.B) * ((tiles + 1) / 2) * pieces >= 256;
}

template <int D, int kX, int kParts>
void weigh_tiles(const Args& A, hipStream_t s) {
  constexpr int kKeys = kWaves * 32 * kX;
  const int chunks = (A.c.cap + kKeys - 1) / kKeys;
  const int heads = A.c.B * A.H, most = (1 << 23) / chunks;
  for (int n0 = 0; n0 < heads; n0 += most) {   // at most 2^23 workgroups a launch
    const int nh = heads - n0 < most ? heads - n0 : most;
    k_weights_tiles<D, kX, kParts><<<unsigned(nh) * unsigned(chunks), kParts * kThreads, 0, s>>>(A, fast_div(uint32_t(chunks)), n0);
  }
}

template <int D>
void attend_chunks(Args& A, hipStream_t s) {
  const unsigned blocks = deal(A, A.slots);
  if (A.c.bs % (512 / D) != 0) k_attend_tiles<D, 1, kWaves><<<blocks, kThreads, 0, s>>>(A);
  else if (eight_waves(A, D)) k_attend_tiles<D, 512 / D, 8><<<blocks, 512, 0, s>>>(A);
  else k_attend_tiles<D, 512 / D, kWaves><<<blocks, kThreads, 0, s>>>(A);
  if (tile_max_pieces(A.c.cap) > 1) {
    const int tiles = first_tile(A.k.n_tokens, A.k.B, A.G);
    k_join_tiles<D><<<dim3(unsigned(tiles) * unsigned(A.H), kRows * D / 1024), kThreads, 0, s>>>(A, fast_div(uint32_t(tiles)));
  }
  if (!A.c.weight) return;
  // A key's sum is the same in all three.  Half as many keys a wave, and of many rows a
  // quarter too, where workgroups of 256 keys do not give every CU two (8 heads of 128, 4
  // rows a token, the whole call, us): 2048 new tokens in 4096 slots, 128 workgroups, 364 : 305 :
  // 215, 128 tokens 49 : 46 in quarters, 64 40.2 : 40.8; 512 over 16384, 512 workgroups, 234 :
  // 242 : 259.
  const bool few = A.c.B * int64_t(A.H) * ((A.c.cap + 255) / 256) < 512;
  if (!few) weigh_tiles<D, 2, 1>(A, s);
  else if (int64_t(A.G) * A.k.max_new < 512) weigh_tiles<D, 1, 1>(A, s);
  else weigh_tiles<D, 1, kRuns>(A, s);
}

}  // namespace

hipError_t launch_attend_tiles(const AttendCall& a, const Partials& places, int slots, hipStream_t s) {
  Args A{};
  A.c = a.c;
  A.k = a.k;
  A.G = a.G;
  A.H = a.c.H;
  A.c_log2 = a.c_log2;
  A.q = a.q, A.out = a.out;
  A.lse = a.lse;
  A.most = tile_max_pieces(a.c.cap);
  A.places = places;
  A.slots = slots;
  if (a.c.D == 128) attend_chunks<128>(A, s);
  else attend_chunks<64>(A, s);
  return hipGetLastError();
}

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
  const bool eight = eight_waves(int64_t(k.n_tokens) * G, k.B, H, D);
  const unsigned blocks = deal(A, first_tile(k.n_tokens, k.B, G, eight ? 2 * kRows : kRows));
  if (eight) k_attend_tiles<128, 0, 8><<<blocks, 512, 0, s>>>(A);
  else if (D == 128) k_attend_tiles<128, 0, kWaves><<<blocks, kThreads, 0, s>>>(A);
  else k_attend_tiles<64, 0, kWaves><<<blocks, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kvc
