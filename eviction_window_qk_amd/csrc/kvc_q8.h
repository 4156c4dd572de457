// 8-bit paged cache: declarations shared by its kernels and host code, and the
// device code that turns values into codes and back.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// Quotient by a divisor known at launch: q = (mulhi(x, m) + x) >> s, exact for
// 0 <= x < 2^31 (m = floor(2^32 (2^s - d) / d) + 1, s = ceil(log2 d)); Granlund and
// Montgomery, Division by Invariant Integers using Multiplication, 1994.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
  return FastDiv{d, uint32_t(m), s};
}

__host__ __device__ __forceinline__ uint32_t quot(FastDiv f, uint32_t x) {
  return uint32_t(((uint64_t(x) * f.m) >> 32) + x) >> f.s;
}

// The same for any 32-bit x.
__device__ __forceinline__ uint32_t quot32(FastDiv f, uint32_t x) {
  const uint32_t hi = __umulhi(x, f.m);
  return f.s == 0 ? x : (((x - hi) >> 1) + hi) >> (f.s - 1);
}

// A cache after validation.
struct Q8 {
  int B, H, D, bs, tb, cap, fmt;
  uint32_t n_blocks;
  FastDiv div;  // by bs
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;
  const int32_t* seq_len;
};

__device__ __forceinline__ int q8_len(const Q8& c, int b) {
  const int len = c.seq_len[b];
  return len < 0 ? 0 : (len < c.cap ? len : c.cap);
}

// Page of logical block j of sequence b, or -1.
__device__ __forceinline__ int q8_page(const Q8& c, int b, int j) {
  const int32_t p = c.table[size_t(b) * c.tb + j];
  return uint32_t(p) < c.n_blocks ? p : -1;
}

// Keys per workgroup of the attention, for a sequence of len keys and R query
// rows: pieces of at most 512 keys (640 for more than 16 rows, whose partial
// sums weigh twice as much), doubled to 2048 while there are more than 64; equal
// pieces, in multiples of the workgroup's 128-key stride.  Shorter pieces keep
// a small batch's latency down, longer ones spend less on starting and joining:
// 8 heads of 4096 keys take 12 us with 512 and 15 with 1024, 512 heads of 4096
// keys 110 and 106; 32 rows on 32 heads of 4096 keys 20 us with 640 and 22 with
// 1024, on 128 heads of 16384 keys 145 and 128.  The length depends on the
// sequence's own length and rows only, so a head's sums are taken in the same
// order whatever else is in the launch.
constexpr int kQ8MaxChunk = 2048;  // the workgroup's LDS holds as many keys
constexpr int kQ8Chunk = 512, kQ8ChunkRows = 640;
static_assert(kQ8Chunk % 128 == 0 && kQ8ChunkRows % 128 == 0 && kQ8MaxChunk % 128 == 0 &&
                  kQ8Chunk <= kQ8MaxChunk && kQ8ChunkRows <= kQ8MaxChunk,
              "pieces are whole strides and fit the LDS");
__host__ __device__ inline int q8_chunk(int len, int rows) {
  int c = rows <= 16 ? kQ8Chunk : kQ8ChunkRows;
  while (c < kQ8MaxChunk && len > 64 * c) c = 2 * c < kQ8MaxChunk ? 2 * c : kQ8MaxChunk;
  const int pieces = (len + c - 1) / c;
  return pieces > 1 ? ((len + pieces - 1) / pieces + 127) & ~127 : c;
}
// The longest piece that any length up to cap has.
inline int q8_longest_chunk(int cap, int rows) {
  const int base = rows <= 16 ? kQ8Chunk : kQ8ChunkRows;
  return cap <= 64 * base ? base : kQ8MaxChunk;
}
// The most pieces that any length up to cap is cut into.
inline int q8_max_pieces(int cap, int rows) {
  const int base = rows <= 16 ? kQ8Chunk : kQ8ChunkRows;
  if (cap <= 64 * base) return cap > 0 ? (cap + base - 1) / base : 1;
  const int n = (cap + kQ8MaxChunk - 1) / kQ8MaxChunk;
  return n > 64 ? n : 64;
}

hipError_t launch_q8_store(const Q8& c, int T, int TS, const int32_t* kept, int n_kept,
                           const void* k, const void* v, hipStream_t s);
hipError_t launch_q8_load(const Q8& c, int T, int TS, void* k_out, void* v_out, hipStream_t s);
hipError_t launch_q8_append(const Q8& c, int W, const int32_t* n_new, const void* k_new,
                            const void* v_new, hipStream_t s);
hipError_t launch_q8_attend(const Q8& c, int G, int W, float c_log2, const void* q, void* out,
                            float* lse, float* part, hipStream_t s);

}  // namespace kvc
