// Page tables on gfx950: allocation, forks, frees, copies and compaction of the
// pages of a paged cache, all decided on the device.
//
// A page is free when its count is zero, and new pages are the lowest free
// ones: there is no free list to keep in step, and the same calls give the
// same tables.  A first launch decides: workgroups list the free pages of their
// tile of the pool in order, others look at the requests; a second applies the
// decisions, table rows by some workgroups and page bytes by others.  A tile's
// rank needs the counts of the tiles before it, which each workgroup takes
// itself from pools of up to 65536 pages; larger pools, and calls for more than
// 4096 sequences, spend a launch on sums first (a launch costs a call about 3 us;
// deciding takes 3 us in a pool of 1000 pages and 7 in one of 32768).  Counts
// change by integer atomics, whose order does not matter to the result.  The
// page copies are bound by HBM (5 TB/s), the rest by launch latency.
#include "kvc_pages.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;    // of the launches that apply
constexpr int kPlanThreads = 1024;  // of those that decide
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPerLane = kPageTile / kPlanThreads;  // pages a lane looks at
enum { kRefused = 0, kShared = 1, kCopied = 2 };    // what a fork pair does

__device__ __forceinline__ int below(uint64_t mask, int lane) {
  return __popcll(mask & ((uint64_t(1) << lane) - 1));
}

// Sum over the workgroup's WAVES waves, in every thread.
template <int WAVES, class T>
__device__ __forceinline__ T block_sum(T x, T* sh) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) x += sh[w];
  return x;
}

// Exclusive prefix sum over the workgroup's threads; *total in every thread.
template <int WAVES, class T>
__device__ __forceinline__ T block_scan(T x, T* sh, T* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T incl = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T y = __shfl_up(incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();
  if (lane == 63) sh[wave] = incl;
  __syncthreads();
  T base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    base += w < wave ? sh[w] : 0;
    all += sh[w];
  }
  *total = all;
  return base + incl - x;
}

// One tile's pages in order: each wave has its share, 64 pages a step.  Bit i
// of the result: the lane's page of step i has a count above zero.
__device__ __forceinline__ uint32_t tile_live(const int32_t* refs, int n, int tile, int* first) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  *first = tile * kPageTile + wave * (kPageTile / kPlanWaves) + lane;
  int r[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {  // no branches: all loads in flight at once
    const int id = *first + i * 64;
    r[i] = refs[id < n ? id : n - 1];
  }
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    live |= r[i] > 0 && *first + i * 64 < n ? 1u << i : 0u;
  return live;
}

// A pool of at most 65536 pages as one workgroup sees it: bit j of a thread's
// mask is page j * 1024 + thread.
constexpr int kOwnTiles = 64 * kPlanThreads / kPageTile, kBatch = 16;
__device__ __forceinline__ uint64_t pool_live(const int32_t* refs, int n) {
  uint64_t mask = 0;
  for (int base = 0; base < n; base += kBatch * kPlanThreads) {
    int r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int id = base + i * kPlanThreads + int(threadIdx.x);
      r[i] = refs[id < n ? id : n - 1];
    }
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      bits |= r[i] > 0 && base + i * kPlanThreads + int(threadIdx.x) < n ? 1u << i : 0u;
    mask |= uint64_t(bits) << (base / kPlanThreads);
  }
  return mask;
}
// This thread's live pages below page `end` of such a mask.
__device__ __forceinline__ int live_in(uint64_t mask, int end) {
  const int k = (end - int(threadIdx.x) + kPlanThreads - 1) / kPlanThreads;
  return k <= 0 ? 0 : __popcll(k >= 64 ? mask : mask & ((uint64_t(1) << k) - 1));
}

// Live pages of each tile, one workgroup each; count is NULL where the tiles
// are few enough to be counted by everybody.
__global__ __launch_bounds__(kPlanThreads) void k_count(Pages t, int32_t* count) {
  __shared__ int sh[kPlanWaves];
  int first;
  const uint32_t live = tile_live(t.refs, t.n, blockIdx.x, &first);
  const int total = block_sum<kPlanWaves>(int(__popc(live)), sh);
  if (threadIdx.x == 0) count[blockIdx.x] = total;
}

// Sum of the first `tiles` tile counts.
__device__ __forceinline__ int counted(const int32_t* count, int tiles, int* sh) {
  int x = 0;
  for (int i = threadIdx.x; i < tiles; i += kPlanThreads) x += count[i];
  return block_sum<kPlanWaves>(x, sh);
}

// Writes the tile's free pages to list[rank]; the last tile also the number of
// all to meta[0].
__device__ __forceinline__ void list_free(const Pages& t, int tile, const int32_t* count,
                                          int32_t* list, int32_t* meta, int* sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int first;
  const uint32_t live = tile_live(t.refs, t.n, tile, &first);
  int before = 0;
  if (count)
    before = counted(count, tile, sh);
  else if (tile > 0)
    before = block_sum<kPlanWaves>(int(__popcll(pool_live(t.refs, tile * kPageTile))), sh);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    mine += __popcll(__ballot(first + i * 64 < t.n && !(live >> i & 1)));
  __syncthreads();
  if (lane == 0) sh[wave] = mine;
  __syncthreads();
  int rank = tile * kPageTile - before, all = rank;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    rank += w < wave ? sh[w] : 0;
    all += sh[w];
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const bool free = first + i * 64 < t.n && !(live >> i & 1);
    const uint64_t m = __ballot(free);
    if (free) list[rank + below(m, lane)] = first + i * 64;
    rank += __popcll(m);
  }
  if ((tile + 1) * int64_t(kPageTile) >= t.n && threadIdx.x == 0) meta[0] = all;
}

__device__ __forceinline__ bool is_page(const Pages& t, int32_t p) {
  return uint32_t(p) < uint32_t(t.n);
}

// --- alloc -------------------------------------------------------------------

// Entries that a sequence's want covers, or -1 when it is refused.
__device__ __forceinline__ int wanted(const Pages& t, int32_t want) {
  if (want < 0 || int64_t(want) > int64_t(t.tb) * t.bs) return -1;
  return int((int64_t(want) + t.bs - 1) / t.bs);
}

// Free pages of a tile each, and the entries that four sequences each miss.
__global__ __launch_bounds__(kPlanThreads) void k_alloc_plan(Pages t, int n_tiles,
                                                             const int32_t* want,
                                                             const int32_t* count, int32_t* list,
                                                             int32_t* meta, int32_t* need) {
  __shared__ int sh[kPlanWaves];
  if (int(blockIdx.x) < n_tiles) return list_free(t, blockIdx.x, count, list, meta, sh);
  const int part = threadIdx.x / kThreads, at = threadIdx.x % kThreads;
  const int b = (int(blockIdx.x) - n_tiles) * (kPlanThreads / kThreads) + part;
  int miss = 0;
  if (b < t.B) {
    const int entries = wanted(t, want[b]);
    const int32_t* row = t.table + size_t(b) * t.tb;
#pragma unroll 8
    for (int j = at; j < entries; j += kThreads) miss += is_page(t, row[j]) ? 0 : 1;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) miss += __shfl_xor(miss, off);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = miss;
  __syncthreads();
  if (at == 0 && b < t.B) {
    miss = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) miss += sh[part * (kThreads / 64) + w];
    need[b] = miss;
  }
}

// need[b] summed over the sequences before each; a sum past 2^31 - 1 stays
// there.
__global__ __launch_bounds__(kPlanThreads) void k_alloc_scan(Pages t, const int32_t* need,
                                                             int32_t* offset) {
  __shared__ int64_t sh[kPlanWaves];
  int64_t base = 0;
  for (int b0 = 0; b0 < t.B; b0 += kPlanThreads) {
    const int b = b0 + int(threadIdx.x);
    int64_t total;
    const int64_t at = base + block_scan<kPlanWaves>(int64_t(b < t.B ? need[b] : 0), sh, &total);
    if (b < t.B) offset[b] = at < 0x7fffffff ? int32_t(at) : 0x7fffffff;
    base += total;
  }
}

// One sequence each; offset is NULL where every workgroup sums for itself.
__global__ __launch_bounds__(kThreads) void k_alloc_apply(Pages t, const int32_t* want,
                                                          const int32_t* list, const int32_t* meta,
                                                          const int32_t* need, const int32_t* offset,
                                                          int32_t* status) {
  __shared__ int sh[kThreads / 64];
  __shared__ int64_t sums[kThreads / 64];
  const int b = blockIdx.x;
  const int entries = wanted(t, want[b]), n = need[b];
  if (n == 0) {  // the same for the whole workgroup
    if (threadIdx.x == 0) status[b] = entries < 0 ? 2 : 0;
    return;
  }
  int64_t off = 0;
  if (offset) {
    off = offset[b];
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < b; i += kThreads) off += need[i];
    off = block_sum<kThreads / 64>(off, sums);
  }
  const bool fits = off + n <= meta[0];
  if (threadIdx.x == 0) status[b] = fits ? 0 : 1;
  if (!fits) return;
  int32_t* row = t.table + size_t(b) * t.tb;
  int rank = int(off);
  for (int j0 = 0; j0 < entries; j0 += kThreads) {
    const int j = j0 + int(threadIdx.x);
    const bool miss = j < entries && !is_page(t, row[j]);
    int total;
    const int at = block_scan<kThreads / 64>(miss ? 1 : 0, sh, &total);
    if (miss) {
      const int32_t p = list[rank + at];
      row[j] = p;
      t.refs[p] = 1;
    }
    rank += total;
  }
}

// A small call in one launch, by one workgroup: the same decisions, with the
// free pages and the needs in LDS; a wave looks at a sequence at a time.
constexpr int kSmallSeqs = 64;
__global__ __launch_bounds__(kPlanThreads) void k_alloc_small(Pages t, const int32_t* want,
                                                              int32_t* status) {
  __shared__ int sh[kPlanWaves];
  __shared__ int32_t list[kPageTile];
  __shared__ int32_t need[kSmallSeqs];  // then the requests before each
  __shared__ int32_t n_free;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int b = wave; b < t.B; b += kPlanWaves) {
    const int entries = wanted(t, want[b]);
    const int32_t* row = t.table + size_t(b) * t.tb;
    int miss = 0;
    for (int j0 = 0; j0 < entries; j0 += 64)
      miss += __popcll(__ballot(j0 + lane < entries && !is_page(t, row[j0 + lane])));
    if (lane == 0) need[b] = miss;
  }
  list_free(t, 0, nullptr, list, &n_free, sh);
  __syncthreads();
  const int b0 = threadIdx.x;
  const int mine = b0 < t.B ? need[b0] : 0;
  int total;
  const int off = block_scan<kPlanWaves>(mine, sh, &total);
  const int free = n_free;
  const bool fits = off + mine <= free;
  __syncthreads();
  if (b0 < t.B) {
    need[b0] = mine > 0 && fits ? off : -1;
    status[b0] = wanted(t, want[b0]) < 0 ? 2 : (fits || mine == 0 ? 0 : 1);
  }
  __syncthreads();
  for (int b = wave; b < t.B; b += kPlanWaves) {
    int rank = need[b];
    if (rank < 0) continue;
    const int entries = wanted(t, want[b]);
    int32_t* row = t.table + size_t(b) * t.tb;
    for (int j0 = 0; j0 < entries; j0 += 64) {
      const bool miss = j0 + lane < entries && !is_page(t, row[j0 + lane]);
      const uint64_t m = __ballot(miss);
      if (miss) {
        const int32_t p = list[rank + below(m, lane)];
        row[j0 + lane] = p;
        t.refs[p] = 1;
      }
      rank += __popcll(m);
    }
  }
}

// --- copies ------------------------------------------------------------------

// One chunk of page `from` to page `to`, in the buffer the chunk belongs to.
// The copy is not read again soon, the page may be: one prompt's open page goes
// to many forks.  With the stores alone past the cache 512 forks of 64 pages
// took 43 us, with loads and stores 62 to 70, with neither 65.
__device__ __forceinline__ void copy_chunk(const Buffers& f, uint32_t chunk, int from, int to) {
  int i = 0;
  while (i + 1 < f.n && chunk >= f.b[i + 1].first) ++i;
  const int64_t at = int64_t(chunk - f.b[i].first) * kCopyChunk;
  const int64_t left = f.b[i].bytes - at;
  const int size = int(left < kCopyChunk ? left : kCopyChunk);
  const char* src = f.b[i].base + int64_t(from) * f.b[i].bytes + at;
  char* dst = f.b[i].base + int64_t(to) * f.b[i].bytes + at;
  if (f.b[i].unit == 16) {
    const u32x4* a = reinterpret_cast<const u32x4*>(src);
    u32x4* z = reinterpret_cast<u32x4*>(dst);
    const int n = size / 16, e = threadIdx.x;
    u32x4 x, y;
    if (e < n) x = a[e];
    if (e + kThreads < n) y = a[e + kThreads];
    if (e < n) __builtin_nontemporal_store(x, z + e);
    if (e + kThreads < n) __builtin_nontemporal_store(y, z + e + kThreads);
  } else if (f.b[i].unit >= 4) {
    for (int e = threadIdx.x; e < size / 4; e += kThreads)
      reinterpret_cast<uint32_t*>(dst)[e] = reinterpret_cast<const uint32_t*>(src)[e];
  } else {
    for (int e = threadIdx.x; e < size; e += kThreads) dst[e] = src[e];
  }
}

__global__ __launch_bounds__(kThreads) void k_pages_copy(int n, int n_pairs, const int32_t* src,
                                                         const int32_t* dst, Buffers f) {
  const uint64_t items = uint64_t(n_pairs) * f.chunks;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = int(it / f.chunks);
    const int32_t from = src[i], to = dst[i];
    if (uint32_t(from) < uint32_t(n) && uint32_t(to) < uint32_t(n) && from != to)
      copy_chunk(f, uint32_t(it % f.chunks), from, to);
  }
}

// --- fork --------------------------------------------------------------------

__device__ __forceinline__ bool is_seq(const Pages& t, int32_t b) {
  return uint32_t(b) < uint32_t(t.B);
}

__device__ __forceinline__ int length_of(const Pages& t, int b) {
  const int len = t.seq_len[b], cap = t.tb * t.bs;
  return len < 0 ? 0 : (len < cap ? len : cap);
}

// Free pages of a tile each, and in the last workgroup what every pair does and
// which of the new pages it takes.
__global__ __launch_bounds__(kPlanThreads) void k_fork_plan(Pages t, int n_tiles, int n_pairs,
                                                            const int32_t* src, const int32_t* dst,
                                                            const int32_t* count, int32_t* list,
                                                            int32_t* meta, int32_t* mark,
                                                            int32_t* kind, int32_t* rank,
                                                            int32_t* from) {
  __shared__ int sh[kPlanWaves];
  if (int(blockIdx.x) < n_tiles) return list_free(t, blockIdx.x, count, list, meta, sh);
  // mark[b]: the first pair whose dst is b
  for (int b = threadIdx.x; b < t.B; b += kPlanThreads)
    __hip_atomic_store(&mark[b], 0x7fffffff, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  for (int i = threadIdx.x; i < n_pairs; i += kPlanThreads)
    if (is_seq(t, dst[i])) atomicMin(&mark[dst[i]], i);
  __syncthreads();
  int base = 0;
  for (int i0 = 0; i0 < n_pairs; i0 += kPlanThreads) {
    const int i = i0 + int(threadIdx.x);
    int what = kRefused, page = -1;
    if (i < n_pairs) {
      const int32_t a = src[i], z = dst[i];
      auto first = [&](int b) {
        return __hip_atomic_load(&mark[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      if (is_seq(t, a) && is_seq(t, z) && first(z) == i && first(a) == 0x7fffffff) {
        const int len = length_of(t, a), whole = len / t.bs;
        what = kShared;
        if (len % t.bs) {
          page = t.table[size_t(a) * t.tb + whole];
          if (is_page(t, page)) what = kCopied;
        }
      }
    }
    int total;
    const int r = base + block_scan<kPlanWaves>(what == kCopied ? 1 : 0, sh, &total);
    if (i < n_pairs) {
      kind[i] = what;
      rank[i] = r;
      from[i] = page;
    }
    base += total;
  }
}

// The first n_rows workgroups write one pair's table row each, the others copy
// page chunks.
__global__ __launch_bounds__(kThreads) void k_fork_apply(Pages t, int n_pairs, int n_rows,
                                                         const int32_t* src, const int32_t* dst,
                                                         const int32_t* kind, const int32_t* rank,
                                                         const int32_t* from, const int32_t* list,
                                                         const int32_t* meta, int32_t* status,
                                                         Buffers f) {
  const int n_free = meta[0];
  if (int(blockIdx.x) < n_rows) {
    const int i = blockIdx.x, what = kind[i];
    const bool fits = what != kCopied || rank[i] < n_free;
    if (threadIdx.x == 0) status[i] = what == kRefused ? 2 : (fits ? 0 : 1);
    if (what == kRefused || !fits) return;
    const int a = src[i], z = dst[i], len = length_of(t, a), whole = len / t.bs;
    const int32_t* ra = t.table + size_t(a) * t.tb;
    int32_t* rz = t.table + size_t(z) * t.tb;
    for (int j = threadIdx.x; j < t.tb; j += kThreads) {
      const int32_t was = rz[j];
      int32_t now = j < whole ? ra[j] : -1;
      if (is_page(t, now)) {
        atomicAdd(&t.refs[now], 1);
      } else {
        now = -1;
      }
      if (j == whole && what == kCopied) {
        now = list[rank[i]];
        t.refs[now] = 1;
      }
      if (is_page(t, was)) atomicSub(&t.refs[was], 1);
      rz[j] = now;
    }
    if (threadIdx.x == 0) t.seq_len[z] = len;
    return;
  }
  const uint64_t items = uint64_t(n_pairs) * f.chunks;
  for (uint64_t it = blockIdx.x - n_rows; it < items; it += gridDim.x - n_rows) {
    const int i = int(it / f.chunks);
    if (kind[i] == kCopied && rank[i] < n_free)
      copy_chunk(f, uint32_t(it % f.chunks), from[i], list[rank[i]]);
  }
}

// --- free --------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void k_pages_free(Pages t, const int32_t* ids) {
  const int32_t b = ids[blockIdx.x];
  if (!is_seq(t, b)) return;
  int32_t* row = t.table + size_t(b) * t.tb;
  // the exchange hands each entry to one workgroup where an id is named twice
  for (int j = threadIdx.x; j < t.tb; j += kThreads) {
    int32_t p = row[j];
    if (is_page(t, p)) {
      p = atomicExch(&row[j], -1);
      if (is_page(t, p)) atomicSub(&t.refs[p], 1);
    } else if (p != -1) {
      row[j] = -1;
    }
  }
  if (threadIdx.x == 0) t.seq_len[b] = 0;
}

// --- compact -----------------------------------------------------------------

// Free pages below n_live ("holes") and live ones at or past it ("movers"), each
// in ascending order: there are as many of one as of the other.  place[p]: p
// itself, -1 where it is free, -2 - m for the m-th mover.
__global__ __launch_bounds__(kPlanThreads) void k_compact_plan(Pages t, const int32_t* count,
                                                               int32_t* holes, int32_t* movers,
                                                               int32_t* place, int32_t* meta,
                                                               int32_t* n_live_out) {
  __shared__ int sh[kPlanWaves];
  __shared__ int64_t sums[kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tile = blockIdx.x;
  int first;
  const uint32_t live = tile_live(t.refs, t.n, tile, &first);
  int before, n_live, low;  // live pages before this tile, in the pool, and that stay
  if (count) {
    before = counted(count, tile, sh);
    n_live = counted(count, int(gridDim.x), sh);
    const int cut = n_live / kPageTile, at = cut * kPageTile;
    low = counted(count, cut, sh);
    low += block_sum<kPlanWaves>(int(__popcll(pool_live(t.refs + at, n_live - at))), sh);
  } else {
    const uint64_t mask = pool_live(t.refs, t.n);
    const int64_t x = int64_t(__popcll(mask)) << 32 | live_in(mask, tile * kPageTile);
    const int64_t y = block_sum<kPlanWaves>(x, sums);
    before = int(y & 0x7fffffff);
    n_live = int(y >> 32);
    low = block_sum<kPlanWaves>(live_in(mask, n_live), sh);
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) mine += __popcll(__ballot(live >> i & 1));
  __syncthreads();
  if (lane == 0) sh[wave] = mine;
  __syncthreads();
  int rank = before;  // live pages before this step
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) rank += w < wave ? sh[w] : 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int id = first + i * 64;
    const bool on = live >> i & 1;
    const uint64_t m = __ballot(on);
    const int r = rank + below(m, lane);
    if (id < t.n) {
      int32_t to = on ? id : -1;
      if (on && id >= n_live) {
        movers[r - low] = id;
        to = -2 - (r - low);
      }
      if (!on && id < n_live) holes[id - r] = id;
      place[id] = to;
    }
    rank += __popcll(m);
  }
  if (tile == 0 && threadIdx.x == 0) {
    meta[0] = n_live;
    meta[1] = n_live - low;  // moves
    *n_live_out = n_live;
  }
}

// Workgroups below n_rows rewrite tables and counts, the others move pages.
__global__ __launch_bounds__(kThreads) void k_compact_apply(Pages t, int n_rows,
                                                            const int32_t* holes,
                                                            const int32_t* movers,
                                                            const int32_t* place,
                                                            const int32_t* meta,
                                                            int32_t* table_out, int32_t* refs_out,
                                                            int32_t* remap, Buffers f) {
  const int n_live = meta[0], moves = meta[1];
  if (int(blockIdx.x) < n_rows) {
    const size_t entries = size_t(t.B) * t.tb, total = entries + size_t(t.n);
    for (size_t e = size_t(blockIdx.x) * kThreads + threadIdx.x; e < total;
         e += size_t(n_rows) * kThreads) {
      const bool entry = e < entries;
      const int32_t p = entry ? t.table[e] : int32_t(e - entries);
      int32_t to = -1;
      if (is_page(t, p)) {
        to = place[p];
        if (to <= -2) to = holes[-2 - to];
      }
      if (entry) {
        table_out[e] = to;
      } else {
        remap[p] = to;
        // counts: a page that stays or moves brings its own; what nobody
        // comes to is free
        if (to >= 0) refs_out[to] = t.refs[p];
        if (p >= n_live) refs_out[p] = 0;
      }
    }
    return;
  }
  const uint64_t items = uint64_t(moves) * f.chunks;
  for (uint64_t it = blockIdx.x - n_rows; it < items; it += gridDim.x - n_rows) {
    const int i = int(it / f.chunks);
    copy_chunk(f, uint32_t(it % f.chunks), movers[i], holes[i]);
  }
}

constexpr int kOwnSeqs = 4096;    // sequences whose needs every workgroup sums

int tiles_of(const Pages& t) { return (t.n + kPageTile - 1) / kPageTile; }

// The tile counts of a pool of many tiles, or NULL.
const int32_t* counts(const Pages& t, int32_t* count, hipStream_t s) {
  const int tiles = tiles_of(t);
  if (tiles <= kOwnTiles) return nullptr;
  k_count<<<unsigned(tiles), kPlanThreads, 0, s>>>(t, count);
  return count;
}

// Workgroups for a launch's chunks.  7900 moved pages of 32 KB took 107 us with
// at most 8192, 97 with 32768; 65536 cost 5 us where there is nothing to move.
unsigned copy_blocks(uint64_t items) {
  return unsigned(items < 32768 ? items : 32768);
}

}  // namespace

PagesWs pages_ws(const Pages& t, int n_pairs) {
  PagesWs w{};
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = (off + n + 63) & ~size_t(63);  // 256 bytes
    return at;
  };
  w.meta = take(64);
  w.count = take(size_t(tiles_of(t)));
  w.list = take(size_t(t.n));
  w.movers = take(size_t(t.n));
  w.place = take(size_t(t.n));
  w.need = take(size_t(t.B));
  w.offset = take(size_t(t.B));
  w.kind = take(size_t(n_pairs));
  w.rank = take(size_t(n_pairs));
  w.from = take(size_t(n_pairs));
  w.total = off;
  return w;
}

hipError_t launch_pages_alloc(const Pages& t, const int32_t* want, int32_t* status, int32_t* ws,
                              hipStream_t s) {
  const PagesWs w = pages_ws(t, 0);
  const int tiles = tiles_of(t), per = kPlanThreads / kThreads;
  // One launch where a wave has at most four steps of table entries to look at:
  // 7.6 us a call against 10 with two launches (16 sequences of 49 entries; 5.3 us
  // on the GPU either way).  256 sequences of 64 entries would take 12 in one.
  const int steps = ((t.B + kPlanWaves - 1) / kPlanWaves) * ((t.tb + 63) / 64);
  if (tiles == 1 && steps <= 4) {
    static_assert(4 * kPlanWaves <= kSmallSeqs, "the needs fit the LDS");
    k_alloc_small<<<1, kPlanThreads, 0, s>>>(t, want, status);
    return hipGetLastError();
  }
  const int32_t* count = counts(t, ws + w.count, s);
  k_alloc_plan<<<unsigned(tiles + (t.B + per - 1) / per), kPlanThreads, 0, s>>>(
      t, tiles, want, count, ws + w.list, ws + w.meta, ws + w.need);
  int32_t* offset = nullptr;
  if (t.B > kOwnSeqs) {
    offset = ws + w.offset;
    k_alloc_scan<<<1, kPlanThreads, 0, s>>>(t, ws + w.need, offset);
  }
  k_alloc_apply<<<unsigned(t.B), kThreads, 0, s>>>(t, want, ws + w.list, ws + w.meta, ws + w.need,
                                                   offset, status);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const Pages& t, int n_pairs, const int32_t* src, const int32_t* dst,
                             const Buffers* groups, int n_groups, int32_t* status, int32_t* ws,
                             hipStream_t s) {
  const PagesWs w = pages_ws(t, n_pairs);
  const int tiles = tiles_of(t);
  const int32_t* count = counts(t, ws + w.count, s);
  k_fork_plan<<<unsigned(tiles + 1), kPlanThreads, 0, s>>>(
      t, tiles, n_pairs, src, dst, count, ws + w.list, ws + w.meta, ws + w.need, ws + w.kind,
      ws + w.rank, ws + w.from);
  for (int gr = 0; gr < n_groups; ++gr) {
    const int rows = gr == 0 ? n_pairs : 0;
    const unsigned blocks = unsigned(rows) + copy_blocks(uint64_t(n_pairs) * groups[gr].chunks);
    if (blocks == 0) continue;
    k_fork_apply<<<blocks, kThreads, 0, s>>>(t, n_pairs, rows, src, dst, ws + w.kind, ws + w.rank,
                                             ws + w.from, ws + w.list, ws + w.meta, status,
                                             groups[gr]);
  }
  return hipGetLastError();
}

hipError_t launch_pages_free(const Pages& t, int n_ids, const int32_t* ids, hipStream_t s) {
  k_pages_free<<<unsigned(n_ids), kThreads, 0, s>>>(t, ids);
  return hipGetLastError();
}

hipError_t launch_pages_copy(int n_blocks, int n_pairs, const int32_t* src, const int32_t* dst,
                             const Buffers* groups, int n_groups, hipStream_t s) {
  for (int gr = 0; gr < n_groups; ++gr) {
    const unsigned blocks = copy_blocks(uint64_t(n_pairs) * groups[gr].chunks);
    if (blocks == 0) continue;
    k_pages_copy<<<blocks, kThreads, 0, s>>>(n_blocks, n_pairs, src, dst, groups[gr]);
  }
  return hipGetLastError();
}

hipError_t launch_pages_compact(const Pages& t, const Buffers* groups, int n_groups,
                                int32_t* table_out, int32_t* refs_out, int32_t* remap,
                                int32_t* n_live, int32_t* ws, hipStream_t s) {
  const PagesWs w = pages_ws(t, 0);
  const int32_t* count = counts(t, ws + w.count, s);
  k_compact_plan<<<unsigned(tiles_of(t)), kPlanThreads, 0, s>>>(
      t, count, ws + w.list, ws + w.movers, ws + w.place, ws + w.meta, n_live);
  const size_t entries = size_t(t.B) * t.tb + size_t(t.n);
  for (int gr = 0; gr < n_groups; ++gr) {
    size_t rows = gr == 0 ? (entries + 4 * kThreads - 1) / (4 * kThreads) : 0;
    if (rows > 2048) rows = 2048;
    const unsigned blocks =
        unsigned(rows) + copy_blocks(uint64_t(t.n / 2) * groups[gr].chunks);  // at most n/2 moves
    if (blocks == 0) continue;
    k_compact_apply<<<blocks, kThreads, 0, s>>>(t, int(rows), ws + w.list, ws + w.movers,
                                                ws + w.place, ws + w.meta, table_out, refs_out,
                                                remap, groups[gr]);
  }
  return hipGetLastError();
}

}  // namespace kvc
