// bf16 paged cache: declarations shared by its kernels and host code.
#pragma once

#include "kvc_div.h"
#include "kvc_internal.h"

namespace kvc {

// A cache after validation.
struct Paged {
  int B, H, D, bs, tb, cap, room;  // cap: bound on a length; room: tb * bs, a head's stride in weight and pos
  uint32_t n_blocks;
  FastDiv div;  // by bs
  uint16_t* k;
  uint16_t* v;
  const int32_t* table;
  int32_t* seq_len;
  float* weight;
  int32_t* pos;
};

// Rows of tokens, strides in values.
struct Rows {
  uint16_t* p;
  int64_t ts, hs;
};

// New tokens packed by sequence.
struct Chunks {
  const int32_t* starts;
  int B, n_tokens, max_new;
};

// A rotation after validation.
struct RopePlan {
  const double* freq;
  int r;            // rotated values of a row, 0: none
  int interleaved;
  float mscale;
  float sign;       // of the angles
};

__device__ __forceinline__ int paged_len(const Paged& c, int b) {
  const int len = c.seq_len[b];
  return len < 0 ? 0 : (len < c.cap ? len : c.cap);
}

// Page of logical block j of sequence b, or -1.
__device__ __forceinline__ int paged_page(const Paged& c, int b, int j) {
  const int32_t p = c.table[size_t(b) * c.tb + j];
  return uint32_t(p) < c.n_blocks ? p : -1;
}

// Row in the pools of slot t of head h of sequence b, or -1: rows are below 2^32 - 1.
__device__ __forceinline__ int64_t paged_row(const Paged& c, int b, int h, int t) {
  const uint32_t j = quot(c.div, uint32_t(t));
  const int page = paged_page(c, b, int(j));
  return page < 0 ? -1
                  : (int64_t(page) * c.H + h) * c.bs + int64_t(uint32_t(t) - j * uint32_t(c.bs));
}

// First token of sequence b, whatever starts holds.
__device__ __forceinline__ int start_of(const Chunks& k, int b) {
  const int a = k.starts[b];
  return a < 0 ? 0 : (a < k.n_tokens ? a : k.n_tokens);
}

// First token and token count of sequence b, whatever starts holds.
__device__ __forceinline__ int2 chunk_of(const Chunks& k, int b) {
  const int a = start_of(k, b);
  int e = k.starts[b + 1];
  e = e < a ? a : (e < k.n_tokens ? e : k.n_tokens);
  return make_int2(a, e - a < k.max_new ? e - a : k.max_new);
}

// The last b in [0, B) with f(start_of(b), b) <= x (0 if there is none), f ascending in
// both: 64 candidates a step, one for each lane.
template <class F>
__device__ __forceinline__ int last_at_or_below(const Chunks& k, int x, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = k.B;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = lane * step;
    const bool in = i < n && f(start_of(k, lo + i), lo + i) <= x;
    const uint64_t m = __ballot(in);
    const int at = m ? (63 - __builtin_clzll(m)) * step : 0;
    lo += at;
    n = n - at < step ? n - at : step;
  }
  return lo;
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
// Two values as bf16, the first one low, in one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// Values of any finite size.  Weights relative to a reference that lags behind the row's
// maximum, or many of them, may take a sum past fp32 though the mean they stand for is
// finite.  A wave whose sums are not finite takes its keys once more, with weights so
// small that a row's sum stays below 1.  They start kLoudHead binades below the limit, so
// that scores may climb by as many before the reference moves.  What they bring below
// 2^-126 is lost: parts of a result below 2^-85 at most.
constexpr float kSumLimit = 0x1p32f;   // of a lane's sum of a tile, where the reference moves
constexpr int kLoudHead = 8;
struct Loud {
  float limit, lift;   // lift: binades of a row's maximum below 1
};
// For rows whose weights are added up by at most `sums` lanes and tiles, of 2^kLoudKeys keys
// at most each.
constexpr int kLoudKeys = 5;
__device__ __forceinline__ Loud loud_of(int sums) {
  const int e = 33 - __builtin_clz(sums | 1);   // 2^-e * sums < 1/2
  return Loud{__uint_as_float(uint32_t(127 - e) << 23), float(e + kLoudKeys + kLoudHead)};
}

// 0 if all of them are finite, otherwise NaN.
__device__ __forceinline__ float unless_finite(float x, float y, float z, float w) {
  return __builtin_fmaf(x, 0.0f, y * 0.0f) + __builtin_fmaf(z, 0.0f, w * 0.0f);
}

// A mean of values within bf16 that the weights' roundings took past its largest, which
// would round to infinity.
constexpr float kMostBf16 = 0x1.fep127f;
__device__ __forceinline__ float within_bf16(float x) {
  return fabsf(x) > kMostBf16 && fabsf(x) < INFINITY ? copysignf(kMostBf16, x) : x;
}

// Keys per workgroup of the attention of few rows, for a sequence of len slots: pieces of at most
// kFewChunk, doubled to kFewMaxChunk while there are more than 64; equal pieces, in
// multiples of the workgroup's 128-key stride.  A piece depends on the sequence's own
// length only, so a head's sums are taken in the same order whatever else is in the
// launch.  Pieces of 256 or 384 start and join too often in batches, of 1024 leave one
// sequence of some thousand slots on too few CUs.
constexpr int kFewChunk = 512, kFewMaxChunk = 2048;
static_assert(kFewChunk % 128 == 0 && kFewMaxChunk % 128 == 0, "pieces are whole strides");
__host__ __device__ inline int few_chunk(int len) {
  int c = kFewChunk;
  while (c < kFewMaxChunk && len > 64 * c) c *= 2;
  const int pieces = (len + c - 1) / c;
  return pieces > 1 ? ((len + pieces - 1) / pieces + 127) & ~127 : c;
}
// The most pieces that any length up to cap is cut into.
inline int few_max_pieces(int cap) {
  if (cap <= 64 * kFewChunk) return cap > 0 ? (cap + kFewChunk - 1) / kFewChunk : 1;
  const int n = (cap + kFewMaxChunk - 1) / kFewMaxChunk;
  return n > 64 ? n : 64;
}

// Sequences with at most kFewRows rows per KV head (rows: new tokens times group) are
// attended by the kernel for few rows, the others by the one for tiles of kTileRows.
constexpr int kFewRows = 32, kTileRows = 128;

// Pieces that the keys of a sequence with `tiles` row tiles are cut into: about kTileWork
// pairs of a tile and a piece for each KV head (eight heads then fill the chip once, two
// workgroups a CU), pieces of at least kTileSpan keys.  The sequence's own length and row
// count decide.  32 pairs (us, 8 heads of 128, 4 rows a token; 64 : 32): one chunk of 512 tokens over
// 16384 slots 158 : 195, of 128 over 8192 41 : 41, ten of 100 over 8192 277 : 223.  Spans
// of 512 : 1024 : 2048: one chunk of 32 over 4096 slots 30 : 37 : 58, 32 of 64 315 : 275 : 275.
constexpr int kTileWork = 64, kTileSpan = 512;
__host__ __device__ inline int tile_pieces(int len, int tiles) {
  const int most = (len + kTileSpan - 1) / kTileSpan, want = kTileWork / tiles;
  const int n = want < most ? want : most;
  return n < 1 ? 1 : n;
}
// Keys of a piece, whole tiles of 64: the last pieces may be empty.
__host__ __device__ inline int tile_span(int len, int pieces) {
  return ((len + pieces - 1) / pieces + 63) & ~63;
}
inline int tile_max_pieces(int cap) { return tile_pieces(cap, 1); }

// Row tiles of packed sequences, numbered through: those of sequence b start here, and
// floor((s + n) G / 128) - floor(s G / 128) + 1 leaves room for its ceil(n G / 128).
__host__ __device__ inline int first_tile(int start, int b, int G, int rows = kTileRows) {
  return int(int64_t(start) * G / rows) + b;
}
// (piece, row tile) pairs of a head over a cache, numbered through: tiles * pieces <=
// max(kTileWork, tiles), and pieces <= most, tile_max_pieces of the longest length.  Only a
// sequence of more than kFewRows rows has any, so b or the count of so many rows before it,
// whichever is less, bounds those before it.  Either bound alone leaves each sequence
// enough behind those before it, so the lesser of both does.
__host__ __device__ inline int first_slot(int start, int b, int G, int most) {
  const int64_t rows = int64_t(start) * G, some = rows / (kFewRows + 1), n = some < b ? some : b, tiles = rows / kTileRows;
  const int64_t by_work = tiles + (kTileWork + 1) * n, by_len = most * (tiles + n);
  return int(by_work < by_len ? by_work : by_len);
}

// What the pieces of rows leave for their joins, outputs and log2 of the sums of 2^x: a place
// for each row and piece, [head][sequence][...], in the order that its kernel likes.  A
// sequence takes at most `most` places a row, and `each` more than it has rows: kTileWork
// tiles, or kFewRows rows in the pieces of few rows.  Places for kTileRows rows of every
// sequence that may have many, 64 times, were 2.3 GB for 64 chunks of 64 tokens in
// tables of 1024 slots (8 heads of 128, 4 rows a token); now 135 MB.
struct Partials {
  float* part;        // [place][D]
  float* stat;        // [place]
  int64_t total;      // places of a head
  int most, each;
};
__host__ __device__ inline int64_t first_place(const Partials& p, int start, int b, int G) {
  const int64_t rows = int64_t(start) * G, by_len = rows * p.most, by_work = rows + int64_t(p.each) * b;
  return by_work < by_len ? by_work : by_len;
}
// Rows of a KV head whose scores are kept, before sequence b: a sequence has at most `rows` of
// them, and no more than its tokens have.
__host__ __device__ inline int64_t score_rows(int start, int b, int G, int rows) {
  const int64_t by_token = int64_t(start) * G, by_seq = int64_t(rows) * b;
  return by_token < by_seq ? by_token : by_seq;
}

// A call of the attention over the cache.
struct AttendCall {
  Paged c;
  Chunks k;
  int G;
  float c_log2;     // scale * log2(e)
  Rows q, out;
  float* lse;       // [n_tokens][G * H] or NULL
};

// Workspace carve-up, in floats.
struct AttendWs {
  size_t scores, part, stat, lse, total;
  Partials places;
  int few_rows, few_pieces;  // most rows of a head (at most kFewRows) and pieces
  int slots;                 // first_slot behind the last token, 0: no sequence has many rows
  int score_stride;          // keys of a row of scores
};
AttendWs attend_ws(const Paged& c, const Chunks& k, int G);

hipError_t launch_rope(const RopePlan& f, int n_tokens, int heads, int D, const int32_t* positions,
                       const Rows& x, const Rows& y, hipStream_t s);
hipError_t launch_paged_append(const Paged& c, const Chunks& k, const int32_t* positions,
                               const RopePlan& f, int q_heads, const Rows& q, const Rows& q_out,
                               const Rows& k_new, const Rows& v_new, hipStream_t s);
hipError_t launch_paged_attend(const AttendCall& a, float* ws, hipStream_t s);
hipError_t launch_attend_tiles(const AttendCall& a, const Partials& places, int slots, hipStream_t s);
hipError_t launch_prompt_attend(int H, int G, int D, const Chunks& k, float c_log2, const Rows& q,
                                const Rows& k_rows, const Rows& v_rows, const Rows& out,
                                float* lse, hipStream_t s);
size_t evict_ws(const Paged& c, int budget);
hipError_t launch_paged_evict(const Paged& c, const int32_t* seen, int K, int sinks, int recent,
                              int32_t* ws, hipStream_t s);

}  // namespace kvc
