// Eviction from a bf16 paged cache by accumulated attention weight.
//
// Every slot gets a 64-bit key whose order is the order of staying:
//   sinks     11 | 0 (32)        | 2^30 - 1 - position (30)
//   recent    10 | 0 (32)        | position
//   others    01 | weight (32)   | 2^30 - 1 - position
// (a weight's bits, turned so that they order as integers).  A workgroup takes one
// head, each wave a range of its slots, and finds the K-th largest key.  Where at most
// kSingles slots have to go (a decode step), it takes the smallest key that often.
// Otherwise it goes digit by digit, eleven bits at a time, from counts in LDS, until the
// slots that share the digits so far are all needed: three digits hold the class and the
// whole weight.  Then it lists, in ascending order, the given-up slots below K and the
// kept ones from K on: as many of either.  A second kernel moves the rows from these to
// those, the only bytes that have to move.
//
// Positions of a head are distinct, so keys are; should they not be, equal keys stay in
// the order of their slots, and both lists still have the same length.
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kSingles = 4, kBits = 11, kBins = 1 << kBits;
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
  if (int(threadIdx.x & 63) == __builtin_ctzll(all)) atomicAdd(&bins[first], __builtin_popcountll(same));
  if (in && bin != first) atomicAdd(&bins[bin], 1);
}

// The smaller of two keys, of equal ones that of the later slot.
__device__ __forceinline__ bool goes_before(uint64_t a, int at, uint64_t b, int bt) {
  return a < b || (a == b && at > bt);
}

// KPT: slots a thread holds in registers, 0: keys are formed again in every pass.
template <int NT, int KPT>
__device__ __forceinline__ void plan(const Evict& E, int n, int b, int len, int* bins) {
  constexpr int kWaves = NT / 64;
  __shared__ int chosen[3];            // digit, slots above it, slots in it
  __shared__ int totals[kWaves][3];    // equal keys, holes, movers of a wave's range
  __shared__ uint64_t low_key[kWaves];
  __shared__ int low_slot[kWaves];
  const Paged& c = E.c;
  const int K = E.K, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float* w = c.weight + size_t(n) * c.room;
  const int32_t* pos = c.pos + size_t(n) * c.room;
  const int64_t recent_from = int64_t(E.seen[b]) - E.recent;
  const int span = ((len + kWaves - 1) / kWaves + 63) & ~63;   // at most KPT * 64
  const int lo = wave * span, hi = lo + span < len ? lo + span : len;
  uint64_t held[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int t = lo + i * 64 + lane;
      held[i] = t < hi ? key_of(w[t], pos[t], E.sinks, recent_from) : 0;   // keys are above 0
    }
  }
  // f(slot, in, key) for the wave's slots, 64 at a time
  auto each = [&](auto f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (lo + i * 64 < hi) f(lo + i * 64 + lane, lo + i * 64 + lane < hi, held[i]);
    } else {
      for (int t = lo; t < hi; t += 64) {
        const bool in = t + lane < hi;
        f(t + lane, in, in ? key_of(w[t + lane], pos[t + lane], E.sinks, recent_from) : 0);
      }
    }
  };

  // Keys from `cut` on stay once shifted by `shift`, of those equal to it `need` do.
  uint64_t cut = 0;
  int shift = 0, need = 0;
  if (len - K <= kSingles) {
    uint64_t last = 0;
    int last_slot = 0x7fffffff;
    for (int m = 0; m < len - K; ++m) {
      uint64_t key = ~uint64_t(0);
      int slot = -1;
      each([&](int t, bool in, uint64_t x) {
        if (in && goes_before(last, last_slot, x, t) && goes_before(x, t, key, slot)) key = x, slot = t;
      });
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor(key, off);
        const int os = __shfl_xor(slot, off);
        if (goes_before(o, os, key, slot)) key = o, slot = os;
      }
      if (lane == 0) low_key[wave] = key, low_slot[wave] = slot;
      __syncthreads();
      key = low_key[0], slot = low_slot[0];
#pragma unroll
      for (int i = 1; i < kWaves; ++i)
        if (goes_before(low_key[i], low_slot[i], key, slot)) key = low_key[i], slot = low_slot[i];
      __syncthreads();
      last = key, last_slot = slot;
    }
    // Slots of the last one's key that are not past it stay.
    cut = last;
    int equal = 0;
    each([&](int t, bool in, uint64_t x) {
      equal += __builtin_popcountll(__ballot(in && x == cut && t < last_slot));
    });
    if (lane == 0) totals[wave][0] = equal;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) need += totals[i][0];
    __syncthreads();
  } else {
    need = K;
    shift = 64;
    while (shift > 0) {
      const int bits = shift < kBits ? shift : kBits;
      shift -= bits;
      for (int i = tid; i < kBins; i += NT) bins[i] = 0;
      __syncthreads();
      each([&](int t, bool in, uint64_t x) {
        // (two shifts: one by all 64 bits is none)
        count_bin(bins, int(x >> shift) & ((1 << bits) - 1), in && ((x >> shift) >> bits) == cut);
      });
      __syncthreads();
      if (wave == 0) {   // the digit that the need-th largest has: a run of bins a lane, from the top
        constexpr int kRun = kBins / 64;
        int sum = 0;
#pragma unroll 8
        for (int i = 0; i < kRun; ++i) sum += bins[kBins - 1 - (kRun * lane + i)];
        int above = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int o = __shfl_up(above, off);
          above += lane >= off ? o : 0;
        }
        above -= sum;    // in the bins of the lanes before
        if (above < need && above + sum >= need) {   // one lane's
          int i = kBins - 1 - kRun * lane;
          while (above + bins[i] < need) above += bins[i--];
          chosen[0] = i;
          chosen[1] = above;
          chosen[2] = bins[i];
        }
      }
      __syncthreads();
      cut = (cut << bits) | uint64_t(chosen[0]);
      need -= chosen[1];
      const bool all = chosen[2] == need;
      __syncthreads();   // before the bins and the choice are written again
      if (all) break;
    }
  }

  // Each wave counts in its range, and writes its part of the lists.
  int equal = 0;
  each([&](int t, bool in, uint64_t x) { equal += __builtin_popcountll(__ballot(in && (x >> shift) == cut)); });
  if (lane == 0) totals[wave][0] = equal;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < wave; ++i) before += totals[i][0];
  const uint64_t below = (uint64_t(1) << lane) - 1;
  auto stays = [&](bool in, uint64_t x, int& eq) {   // eq: equal keys before these 64 slots
    x >>= shift;
    const uint64_t m = __ballot(in && x == cut);
    const bool yes = in && (x > cut || (x == cut && eq + __builtin_popcountll(m & below) < need));
    eq += __builtin_popcountll(m);
    return yes;
  };
  int eq = before, holes = 0, movers = 0;
  each([&](int t, bool in, uint64_t x) {
    const bool yes = stays(in, x, eq);
    holes += __builtin_popcountll(__ballot(in && !yes && t < K));
    movers += __builtin_popcountll(__ballot(yes && t >= K));
  });
  if (lane == 0) totals[wave][1] = holes, totals[wave][2] = movers;
  __syncthreads();
  int hole0 = 0, mover0 = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < wave) hole0 += totals[i][1], mover0 += totals[i][2];
    total += totals[i][2];
  }
  eq = before;
  int32_t* const to = E.to + size_t(n) * E.most;
  int32_t* const from = E.from + size_t(n) * E.most;
  each([&](int t, bool in, uint64_t x) {
    const bool yes = stays(in, x, eq), hole = in && !yes && t < K, mover = yes && t >= K;
    const uint64_t mh = __ballot(hole), mm = __ballot(mover);
    if (hole) to[hole0 + __builtin_popcountll(mh & below)] = t;
    if (mover) from[mover0 + __builtin_popcountll(mm & below)] = t;
    hole0 += __builtin_popcountll(mh);
    mover0 += __builtin_popcountll(mm);
  });
  if (tid == 0) E.count[n] = total;
}

template <int NT>
__global__ __launch_bounds__(NT) void k_evict_plan(Evict E) {
  __shared__ int bins[kBins];
  const int n = blockIdx.x, b = n / E.c.H, len = paged_len(E.c, b);
  if (len <= E.K) {
    if (threadIdx.x == 0) E.count[n] = 0;
  } else if (len <= 4 * NT) {
    plan<NT, 4>(E, n, b, len, bins);
  } else if (len <= 16 * NT) {
    plan<NT, 16>(E, n, b, len, bins);
  } else {
    plan<NT, 0>(E, n, b, len, bins);
  }
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
  // By the longest length there can be: few waves meet sooner.
  if (c.cap <= 2048) k_evict_plan<256><<<unsigned(heads), 256, 0, s>>>(E);
  else k_evict_plan<1024><<<unsigned(heads), 1024, 0, s>>>(E);
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
