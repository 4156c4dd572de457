// Eviction from a bf16 paged cache by accumulated attention weight.
//
// Every slot gets a 64-bit key whose order is the order of staying:
//   sinks     11 | 0 (32)        | 2^30 - 1 - position (30)
//   recent    10 | 0 (32)        | position
//   others    01 | weight (32)   | 2^30 - 1 - position
// (a weight's bits, turned so that they order as integers).  A workgroup takes one
// head and finds the K-th largest key.  Where at most kSingles slots have to go (a decode
// step), it takes the smallest key that often.  Otherwise it goes digit by digit, from
// counts in LDS, until the slots that share the digits so far are all needed.  Digits are
// of 11, 11 and 10 bits, so that none crosses from a key's upper word (the class and
// all but two bits of the weight) into the lower.  Then it lists, in ascending order, the
// given-up slots below K and the kept ones from K on, as many of either: a thread takes
// neighbouring slots, and a sum over the workgroup says where its own begin.  A second
// kernel moves the rows from these to those, the only bytes that have to move.
//
// A page that another entry of the table names too (a fork's) is not written: entries in use
// are counted page by page, and a sequence that would write to a page counted twice stays as
// it is.  The counts cost a launch before the plan, which starts them at zero.
//
// Positions of a head are distinct, so keys are; should they not be, equal keys stay in
// the order of their slots, and both lists still have the same length.
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
template <class T>
struct __attribute__((packed, aligned(4))) Loose { T v; };  // at any slot

constexpr int kSingles = 4, kBins = 1 << 11, kHeld = 16384;
constexpr int kMoveThreads = 256;
constexpr int kLastPos = (1 << 30) - 1;

struct Evict {
  Paged c;
  const int32_t* seen;
  int K, sinks, recent, most;  // most: moves of a head
  int32_t* count;              // [heads]
  int32_t* from;               // [heads][most]
  int32_t* to;                 // [heads][most]
  int32_t* users;              // [n_blocks] entries that name a page, of pages that any names
};

// f(page) for the pages of sequence b's first `slots` slots, by the threads of a workgroup.
template <class F>
__device__ __forceinline__ void each_page(const Paged& c, int b, int slots, F f) {
  const int n = slots > 0 ? int(quot(c.div, uint32_t(slots - 1))) + 1 : 0;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int page = paged_page(c, b, j);
    if (page >= 0) f(page);
  }
}

__global__ __launch_bounds__(kMoveThreads) void k_evict_users(Evict E) {
  const int b = blockIdx.x;
  each_page(E.c, b, paged_len(E.c, b), [&](int page) { E.users[page] = 0; });
}

__device__ __forceinline__ uint64_t key_of(float w, int pos, int sinks, int64_t recent_from) {
  const uint32_t p = uint32_t(pos < 0 ? 0 : (pos < kLastPos ? pos : kLastPos)), back = kLastPos - p;
  const uint32_t u = w != w ? 0xff800000u : __float_as_uint(w + 0.0f);  // -0 is 0, NaN -inf
  const uint32_t order = u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
  const bool sink = pos < sinks, recent = pos >= recent_from;
  const uint32_t hi = sink ? 3u << 30 : (recent ? 2u << 30 : 1u << 30 | order >> 2);
  const uint32_t lo = sink ? back : (recent ? p : order << 30 | back);
  return uint64_t(hi) << 32 | lo;
}

// The smaller of two keys, of equal ones that of the later slot.
__device__ __forceinline__ bool goes_before(uint64_t a, int at, uint64_t b, int bt) {
  return a < b || (a == b && at > bt);
}

// Place of a tile's key in LDS: neighbouring slots of a thread off the other threads' banks.
__host__ __device__ constexpr int place(int t) { return t + (t >> 4); }

// HELD: all keys of a head fit the LDS (kHeld of them at most); otherwise they are formed
// again in every pass, and lie there for the lists, a tile of kHeld at a time.  Of a
// head of 16384 slots the loads take 5 us (four slots a load, all of a thread's on their way
// at once; one at a time 16), a digit 3.
template <int NT, bool HELD>
__global__ __launch_bounds__(NT) void k_evict_plan(Evict E) {
  constexpr int kWaves = NT / 64;
  extern __shared__ __align__(16) uint64_t held[];
  __shared__ int bins[kBins];
  __shared__ int chosen[3];            // digit, slots above it, slots in it
  __shared__ int totals[kWaves];
  __shared__ uint64_t low_key[kWaves];
  __shared__ int low_slot[kWaves];
  const Paged& c = E.c;
  const int n = blockIdx.x, b = n / c.H, len = paged_len(c, b);
  const int K = E.K, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (n == b * c.H) each_page(c, b, len, [&](int page) { atomicAdd(&E.users[page], 1); });
  if (len <= K) {
    if (tid == 0) E.count[n] = 0;
    return;
  }
  const float* w = c.weight + size_t(n) * c.room;
  const int32_t* pos = c.pos + size_t(n) * c.room;
  const int64_t recent_from = int64_t(E.seen[b]) - E.recent;
  // Keys of the slots from t0 on to LDS.
  auto hold = [&](int t0, int count) {
    constexpr int kAhead = 4;
    for (int t = 4 * tid; t < count; t += kAhead * 4 * NT) {
      f32x4 x[kAhead];
      i32x4 p[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int at = t + a * 4 * NT;
        if (at + 3 < count) {
          x[a] = reinterpret_cast<const Loose<f32x4>*>(w + t0 + at)->v;
          p[a] = reinterpret_cast<const Loose<i32x4>*>(pos + t0 + at)->v;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[a][i] = at + i < count ? w[t0 + at + i] : 0.0f;
            p[a][i] = at + i < count ? pos[t0 + at + i] : 0;
          }
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + a * 4 * NT + i < count)
            held[place(t + a * 4 * NT + i)] = key_of(x[a][i], p[a][i], E.sinks, recent_from);
    }
    __syncthreads();
  };
  if (HELD) hold(0, len);
  // f(slot, key) in any order, four keys read ahead
  auto each = [&](auto f) {
    constexpr int kAhead = 4;
    for (int t0 = tid; t0 < len; t0 += kAhead * NT) {
      uint64_t x[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int t = t0 + a * NT;
        x[a] = 0;
        if (t < len) x[a] = HELD ? held[place(t)] : key_of(w[t], pos[t], E.sinks, recent_from);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (t0 + a * NT < len) f(t0 + a * NT, x[a]);
    }
  };
  // Sum over the threads before; all of it in `whole`.
  auto sum_before = [&](int x, int& whole) {
    int sum = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off);
      sum += lane >= off ? o : 0;
    }
    if (lane == 63) totals[wave] = sum;
    __syncthreads();
    sum -= x;
    whole = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const int o = totals[i];
      sum += i < wave ? o : 0;
      whole += o;
    }
    __syncthreads();
    return sum;
  };

  // Which slots stay.  SINGLES: those whose key is past (cut, cut_slot); ALL: those whose
  // shifted key is at least cut; else those past cut and the first `need` of it.
  enum { SINGLES, ALL, SOME } which = SOME;
  uint64_t cut = 0;
  int shift = 64, need = K, cut_slot = 0x7fffffff;
  if (len - K <= kSingles) {
    which = SINGLES;
    for (int m = 0; m < len - K; ++m) {
      uint64_t key = ~uint64_t(0);
      int slot = -1;
      each([&](int t, uint64_t x) {
        if (goes_before(cut, cut_slot, x, t) && goes_before(x, t, key, slot)) key = x, slot = t;
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
      cut = key, cut_slot = slot;
    }
  } else {
    while (shift > 0 && which != ALL) {
      const int bits = (shift & 31) == 10 ? 10 : 11;
      shift -= bits;
      for (int i = tid; i < kBins; i += NT) bins[i] = 0;
      __syncthreads();
      const bool upper = shift >= 32;
      const int by = shift & 31;
      const uint32_t cut_hi = upper ? 0 : uint32_t(cut >> (32 - by - bits));   // the whole upper word, once it is known
      const uint32_t cut_now = upper ? uint32_t(cut) : uint32_t(cut & ((uint64_t(1) << (32 - by - bits)) - 1));
      each([&](int, uint64_t x) {
        const uint32_t word = upper ? uint32_t(x >> 32) : uint32_t(x), digit = word >> by;
        // the digits above in this word: none for the first
        const bool same = by + bits == 32 || (word >> (by + bits)) == cut_now;
        if (same && (upper || uint32_t(x >> 32) == cut_hi)) atomicAdd(&bins[digit & ((1u << bits) - 1)], 1);
      });
      __syncthreads();
      // The digit that the need-th largest has: a run of bins a thread, from the top.
      constexpr int kRun = kBins / NT;
      int mine[kRun], sum = 0, whole;
#pragma unroll
      for (int i = 0; i < kRun; ++i) sum += mine[i] = bins[kBins - 1 - (kRun * tid + i)];
      int above = sum_before(sum, whole);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (above < need && above + mine[i] >= need) {   // one thread's
          chosen[0] = kBins - 1 - (kRun * tid + i);
          chosen[1] = above;
          chosen[2] = mine[i];
        }
        above += mine[i];
      }
      __syncthreads();
      cut = (cut << bits) | uint64_t(chosen[0]);
      need -= chosen[1];
      if (chosen[2] == need) which = ALL;
    }
    if (which == ALL) cut <<= shift;
  }

  int32_t* const to = E.to + size_t(n) * E.most;
  int32_t* const from = E.from + size_t(n) * E.most;
  int equal = 0, n_holes = 0, n_movers = 0;   // of the tiles before: slots of the cut's key, listed ones
  for (int t0 = 0; t0 < len; t0 += kHeld) {
    const int count = len - t0 < kHeld ? len - t0 : kHeld;
    if (!HELD) hold(t0, count);
    const int per = (count + NT - 1) / NT, lo = tid * per, hi = lo + per < count ? lo + per : count;
    uint32_t stay = 0;                 // bit i: slot lo + i; at most kHeld / NT of them
    if (which == SOME) {
      int mine = 0, whole;
      for (int t = lo; t < hi; ++t) mine += held[place(t)] == cut;
      int at = equal + sum_before(mine, whole);
      equal += whole;
      for (int t = lo; t < hi; ++t) {
        const uint64_t x = held[place(t)];
        if (x > cut || (x == cut && at++ < need)) stay |= 1u << (t - lo);
      }
    } else {
#pragma unroll 4
      for (int t = lo; t < hi; ++t) {
        const uint64_t x = held[place(t)];
        const bool yes = which == ALL ? x >= cut : goes_before(cut, cut_slot, x, t0 + t);
        stay |= uint32_t(yes) << (t - lo);
      }
    }
    const int here = hi > lo ? hi - lo : 0, below = K - t0 - lo;     // slots, those below K
    const uint32_t all = (1u << here) - 1, low = below >= here ? all : (below > 0 ? (1u << below) - 1 : 0);
    uint32_t holes = ~stay & low, movers = stay & all & ~low;
    int whole;
    const int before = sum_before(__builtin_popcount(holes) | __builtin_popcount(movers) << 16, whole);
    int h = n_holes + (before & 0xffff), m = n_movers + (before >> 16);
    for (; holes; holes &= holes - 1) to[h++] = t0 + lo + __builtin_ctz(holes);
    for (; movers; movers &= movers - 1) from[m++] = t0 + lo + __builtin_ctz(movers);
    n_holes += whole & 0xffff;
    n_movers += whole >> 16;
    if (!HELD) __syncthreads();        // before the next tile's keys
  }
  if (tid == 0) E.count[n] = n_movers;
}

// A row's 16-byte pieces by D/8 lanes; the lists' slots are disjoint, so the order does
// not matter.  Bound by HBM: 32 heads of 16384 slots cut to 4096 move 98000 rows of 512 bytes
// in 18 to 19 us (100 MB in and out, 5.3 to 5.5 TB/s).
template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_evict_move(Evict E) {
  constexpr int kPieces = D / 8, kAtOnce = kMoveThreads / kPieces;
  const Paged& c = E.c;
  const int n = blockIdx.x, b = n / c.H, h = n - b * c.H;
  const int moves = E.count[n], p = threadIdx.x % kPieces;
  // One workgroup a sequence sets its length, and no other one reads it.
  const bool sets = blockIdx.y == 0 && h == 0 && paged_len(c, b) > E.K;
  if (!sets && int(blockIdx.y) * kAtOnce >= moves) return;
  bool shared = false;
  each_page(c, b, E.K, [&](int page) { shared |= E.users[page] > 1; });
  if (__syncthreads_or(shared)) return;
  if (sets && threadIdx.x == 0) c.seq_len[b] = E.K;
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
  return ((heads * (1 + 2 * size_t(most_moves(c, K))) + c.n_blocks) * 4 + 255) & ~size_t(255);
}

hipError_t launch_paged_evict(const Paged& c, const int32_t* seen, int K, int sinks, int recent,
                              int32_t* ws, hipStream_t s) {
  const int heads = c.B * c.H;
  Evict E{c, seen, K, sinks, recent, most_moves(c, K), ws, nullptr, nullptr, nullptr};
  E.from = ws + heads;
  E.to = E.from + size_t(heads) * E.most;
  E.users = E.to + size_t(heads) * E.most;
  k_evict_users<<<unsigned(c.B), kMoveThreads, 0, s>>>(E);
  // By the longest length there can be: few waves meet sooner.
  const auto lds = [](int slots) { return size_t(place(slots)) * 8; };
  if (c.cap <= 2048) k_evict_plan<256, true><<<unsigned(heads), 256, lds(c.cap), s>>>(E);
  else if (c.cap <= kHeld) k_evict_plan<1024, true><<<unsigned(heads), 1024, lds(c.cap), s>>>(E);
  else k_evict_plan<1024, false><<<unsigned(heads), 1024, lds(kHeld), s>>>(E);
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
