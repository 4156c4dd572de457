// Eviction from a bf16 paged cache by accumulated attention weight.
//
// Every slot gets a 64-bit key whose order is the order of staying:
//   sinks     11 | 0 (32)        | 2^30 - 1 - position (30)
//   recent    10 | 0 (32)        | position
//   others    01 | weight (32)   | 2^30 - 1 - position
// (a weight's bits, turned so that they order as integers).  A workgroup takes one
// head and finds the K-th largest key digit by digit, eight bits at a time, from counts
// in LDS; it is done once the slots that share the digits so far are all needed.
// Then it lists, in ascending order, the given-up slots below K and the kept ones
// from K on: as many of either.  A second kernel moves the rows from these to those,
// the only bytes that have to move.
//
// Positions of a head are distinct, so keys are; should they not be, equal keys stay in
// the order of their slots, and both lists still have the same length.
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMoveThreads = 256;
constexpr int kLastPos = (1 << 30) - 1;

struct Evict {
  Paged c;
  const int32_t* seen;
  int K, sinks, recent, most;  // most: moves of a head
  int32_t* count;              // [heads]
  int32_t* from;               // [heads][most]
  int32_t* to;                 // [heads][most]
};

__device__ __forceinline__ uint64_t key_of(float w, int pos, int sinks, int64_t recent_from) {
  const uint64_t p = uint64_t(pos < 0 ? 0 : (pos < kLastPos ? pos : kLastPos));
  if (pos < sinks) return (uint64_t(3) << 62) | (kLastPos - p);
  if (pos >= recent_from) return (uint64_t(2) << 62) | p;
  const uint32_t u = w != w ? 0xff800000u : __float_as_uint(w + 0.0f);  // -0 is 0, NaN -inf
  const uint32_t order = u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
  return (uint64_t(1) << 62) | (uint64_t(order) << 30) | (kLastPos - p);
}

// One count for each lane's bin; the lanes that share the first one's add theirs in one.
__device__ __forceinline__ void count_bin(int* bins, int bin, bool in) {
  const uint64_t all = __ballot(in);
  if (!all) return;
  const int first = __shfl(bin, __builtin_ctzll(all));
  const uint64_t same = __ballot(in && bin == first);
  if ((threadIdx.x & 63) == __builtin_ctzll(all)) atomicAdd(&bins[first], __builtin_popcountll(same));
  if (in && bin != first) atomicAdd(&bins[bin], 1);
}

__global__ __launch_bounds__(kThreads) void k_evict_plan(Evict E) {
  __shared__ int bins[256];
  __shared__ int chosen[3];            // digit, slots above it, slots in it
  __shared__ int totals[kWaves][3];    // equal keys, holes, movers of a wave's range
  const Paged& c = E.c;
  const int n = blockIdx.x, b = n / c.H, K = E.K;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = paged_len(c, b);
  if (len <= K) {
    if (tid == 0) E.count[n] = 0;
    return;
  }
  const float* w = c.weight + size_t(n) * c.room;
  const int32_t* pos = c.pos + size_t(n) * c.room;
  const int64_t recent_from = int64_t(E.seen[b]) - E.recent;
  auto key = [&](int t) { return key_of(w[t], pos[t], E.sinks, recent_from); };

  // Keys above `prefix` (its digits below `shift` zero) stay, of those that share its
  // digits `need` do.
  uint64_t prefix = 0;
  int shift = 64, need = K;
  while (shift > 0) {
    shift -= 8;
    if (tid < 256) bins[tid] = 0;
    __syncthreads();
    for (int t = wave * 64; t < len; t += kThreads) {   // whole waves
      const int at = t + lane;
      const uint64_t x = at < len ? key(at) : 0;
      const bool in = at < len && (shift == 56 || (x >> (shift + 8)) == (prefix >> (shift + 8)));
      count_bin(bins, int(x >> shift) & 255, in);
    }
    __syncthreads();
    if (wave == 0) {   // the digit that the need-th largest has: four bins a lane, from the top
      int mine[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += mine[i] = bins[255 - 4 * lane - i];
      int above = sum;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(above, off);
        above += lane >= off ? o : 0;
      }
      above -= sum;    // in the bins of the lanes before
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + mine[i] >= need) {
          chosen[0] = 255 - 4 * lane - i;
          chosen[1] = above;
          chosen[2] = mine[i];
        }
        above += mine[i];
      }
    }
    __syncthreads();
    prefix |= uint64_t(chosen[0]) << shift;
    need -= chosen[1];
    const bool all = chosen[2] == need;
    __syncthreads();   // before the bins and the choice are written again
    if (all) break;
  }

  // Each wave takes a range of slots, counts, and writes its part of the lists.
  const int span = ((len + kWaves - 1) / kWaves + 63) & ~63;
  const int lo = wave * span, hi = lo + span < len ? lo + span : len;
  const uint64_t cut = prefix >> shift;
  int equal = 0;
  for (int t = lo; t < hi; t += 64) {
    const int at = t + lane;
    equal += __builtin_popcountll(__ballot(at < hi && (key(at) >> shift) == cut));
  }
  if (lane == 0) totals[wave][0] = equal;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < wave; ++i) before += totals[i][0];
  const uint64_t below = (uint64_t(1) << lane) - 1;
  auto stays = [&](int at, bool in, int& eq) {   // eq: equal keys before this wave's 64 slots
    const uint64_t x = in ? key(at) >> shift : 0;
    const uint64_t m = __ballot(in && x == cut);
    const bool yes = in && (x > cut || (x == cut && eq + __builtin_popcountll(m & below) < need));
    eq += __builtin_popcountll(m);
    return yes;
  };
  int eq = before, holes = 0, movers = 0;
  for (int t = lo; t < hi; t += 64) {
    const int at = t + lane;
    const bool in = at < hi, yes = stays(at, in, eq);
    holes += __builtin_popcountll(__ballot(in && !yes && at < K));
    movers += __builtin_popcountll(__ballot(yes && at >= K));
  }
  if (lane == 0) totals[wave][1] = holes, totals[wave][2] = movers;
  __syncthreads();
  int hole0 = 0, mover0 = 0, total = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < wave) hole0 += totals[i][1], mover0 += totals[i][2];
    total += totals[i][2];
  }
  eq = before;
  for (int t = lo; t < hi; t += 64) {
    const int at = t + lane;
    const bool in = at < hi, yes = stays(at, in, eq);
    const bool hole = in && !yes && at < K, mover = yes && at >= K;
    const uint64_t mh = __ballot(hole), mm = __ballot(mover);
    if (hole) E.to[size_t(n) * E.most + hole0 + __builtin_popcountll(mh & below)] = at;
    if (mover) E.from[size_t(n) * E.most + mover0 + __builtin_popcountll(mm & below)] = at;
    hole0 += __builtin_popcountll(mh);
    mover0 += __builtin_popcountll(mm);
  }
  if (tid == 0) E.count[n] = total;
}

// A row's 16-byte pieces by D/8 lanes; the lists' slots are disjoint, so the order does
// not matter.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_evict_move(Evict E) {
  constexpr int kPieces = D / 8, kAtOnce = kMoveThreads / kPieces;
  const Paged& c = E.c;
  const int n = blockIdx.x, b = n / c.H, h = n - b * c.H;
  const int moves = E.count[n], p = threadIdx.x % kPieces;
  if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) {
    const int len = paged_len(c, b);
    c.seq_len[b] = len < E.K ? len : E.K;
  }
  for (int i = blockIdx.y * kAtOnce + threadIdx.x / kPieces; i < moves; i += gridDim.y * kAtOnce) {
    const int from = E.from[size_t(n) * E.most + i], to = E.to[size_t(n) * E.most + i];
    const int64_t rf = paged_row(c, b, h, from), rt = paged_row(c, b, h, to);
    if (rf >= 0 && rt >= 0) {
      const u32x4 k = *reinterpret_cast<const u32x4*>(c.k + rf * D + p * 8);
      const u32x4 v = *reinterpret_cast<const u32x4*>(c.v + rf * D + p * 8);
      *reinterpret_cast<u32x4*>(c.k + rt * D + p * 8) = k;
      *reinterpret_cast<u32x4*>(c.v + rt * D + p * 8) = v;
    }
    if (p == 0) {
      const size_t row = size_t(n) * c.room;
      c.weight[row + to] = c.weight[row + from];
      c.pos[row + to] = c.pos[row + from];
    }
  }
}

int most_moves(const Paged& c, int K) {
  const int over = c.cap - K;
  return over < 0 ? 0 : (over < K ? over : K);
}

}  // namespace

size_t evict_ws(const Paged& c, int K) {
  const size_t heads = size_t(c.B) * c.H;
  return (heads * (1 + 2 * size_t(most_moves(c, K))) * 4 + 255) & ~size_t(255);
}

hipError_t launch_paged_evict(const Paged& c, const int32_t* seen, int K, int sinks, int recent,
                              int32_t* ws, hipStream_t s) {
  const int heads = c.B * c.H;
  Evict E{c, seen, K, sinks, recent, most_moves(c, K), ws, nullptr, nullptr};
  E.from = ws + heads;
  E.to = E.from + size_t(heads) * E.most;
  k_evict_plan<<<unsigned(heads), kThreads, 0, s>>>(E);
  // About 2048 workgroups where the heads are fewer.
  const int per = kMoveThreads / (c.D / 8), need = (E.most + per - 1) / per;
  int y = heads < 2048 ? 2048 / heads : 1;
  y = y < need ? y : need;
  const dim3 grid{unsigned(heads), unsigned(y < 1 ? 1 : y)};
  if (c.D == 128) k_evict_move<128><<<grid, kMoveThreads, 0, s>>>(E);
  else k_evict_move<64><<<grid, kMoveThreads, 0, s>>>(E);
  return hipGetLastError();
}

}  // namespace kvc
