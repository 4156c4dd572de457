// Attention of a few new tokens per sequence over the bf16 paged cache on gfx950.
//
// For every (sequence, KV head) the G query heads' n new tokens form the R = G*n rows
// (row r: token r / G, head r % G of the group) of two products against the same
// keys and values:
//   x = c * <q, k>,  w = 2^(x - m),  l = sum w,  out = sum w * v / l
// with c = scale * log2(e).  Each cached byte is read once for all R rows; with the few
// rows of a decode step the bound is HBM: 4*d bytes a key.
//
// Both products run on bf16 matrix instructions, 16x16x32, and are taken transposed,
// S' = K Q' and O' = V' P': the lane that holds eight scores of a query row (keys
// 4g..4g+3 of two 16-key tiles, g its 16-lane group) holds exactly the eight weights
// that the second product wants from it, so the weights never leave their lane.  K
// fragments are loaded as they lie in memory; V is read eight keys deep and D/16
// values wide per lane and turned in registers by byte permutes.  Weights enter the
// second product as bf16, their sum is fp32.
//
// m is a reference, not the running maximum: any value serves as long as no sum
// overflows, so a tile is summed against the present one and m moves to the row's maximum
// only when a lane's sum passes 2^32 (the first tile always does).  A wave whose values are
// so large that their sums pass fp32 takes them a second time, with smaller weights (loud_of).
//
// The keys of a head are cut into pieces by its own length (few_chunk); the four
// waves of a piece take its 32-key tiles in turn, and their sums meet in LDS.  A
// workgroup takes one piece, and a second kernel joins the pieces and adds up what each
// slot receives, or it takes a head's few pieces and does both itself (whole_heads).  Where a
// piece's keys are is looked up once, into LDS, four keys at a time where the page size
// is a multiple of four.
//
// Measured (128 values, the kernel alone): 4 rows of 131072 slots of 8 heads 84 us (537 MB,
// 6.4 TB/s), 7 rows of about 1100 slots of 256 heads with their weights, in one launch,
// 33 us (145 MB, 4.4 TB/s): there the start, the join and the weights of a head are a
// quarter of its time, and the next head's loads do not cover them.
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr uint32_t kNone = 0xffffffffu;  // no row: past the end or in no page
constexpr float kFar = 0x1p64f;          // -m of a row that has seen nothing
constexpr int kWholePieces = 3;          // pieces of a head that one workgroup may take

struct Args {
  AttendCall a;
  int pieces, rows;  // of the longest length and the longest chunk: the grid's
  FastDiv by_G, by_pieces, by_H;
  int units;         // (head, piece) pairs of this launch
  int n0;            // its first head
  Partials places;   // of a sequence [row][piece]
  float* scores;     // NULL, or x: [row][score_stride] from first_score on
  int score_stride;
};

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool STREAM, class T>
__device__ __forceinline__ T load(const uint16_t* at) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T*>(at));
  else return *reinterpret_cast<const T*>(at);
}

// Place of the first piece of a head's first row.
__device__ __forceinline__ size_t place_of(const Args& A, int start, int b, int h) {
  return size_t(h) * A.places.total + first_place(A.places, start, b, A.a.G);
}

// A head's first row of scores.
__device__ __forceinline__ float* first_score(const Args& A, int start, int b, int h, int R) {
  return A.scores + (score_rows(start, b, A.a.G, A.rows) * A.a.c.H + h * R) * A.score_stride;
}

// Four output values of row r of a head, and log2 of its sum of 2^x.
__device__ __forceinline__ void finish(const Args& A, int token, int head, int dim, f32x4 out, float b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = within_bf16(out[i]);
  *reinterpret_cast<u32x2*>(A.a.out.p + token * A.a.out.ts + head * A.a.out.hs + dim) =
      u32x2{pack_bf16(out.x, out.y), pack_bf16(out.z, out.w)};
  if (A.a.lse && dim == 0)
    A.a.lse[size_t(token) * (A.a.G * A.a.c.H) + head] = b * 0.6931471805599453f;
}

// What four slots of a head from t on receive from its R rows: the sum down the rows of
// 2^(x - log2 of the row's sum), less: minus these logarithms.  The scores were kept (4
// bytes a row and slot; the keys would be 2 * d bytes a slot again).
__device__ __forceinline__ void weigh_four(const Args& A, const float* scores, int t, int len, int R,
                                           const float* less, const float* was, float* to) {
  const float* x = scores + t;
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll 8
  for (int r = 0; r < R; ++r) {
    const f32x4 y = *reinterpret_cast<const f32x4*>(x + size_t(r) * A.score_stride);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += fast_exp2(y[i] + less[r]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t + i < len && sum[i] > 0.0f) to[i] = was[i] + sum[i];
}

// The head and piece of a workgroup.  Pieces of one head follow each other, each head's
// rotated by one: workgroups go to the XCDs in turn, and where only the first pieces of a
// long table have keys they would all be one XCD's.
__device__ __forceinline__ bool piece_of(const Args& A, int& n, int& piece) {
  const uint32_t unit = blockIdx.x;
  if (unit >= uint32_t(A.units)) return false;
  const int nth = int(quot(A.by_pieces, unit));
  piece = int(unit) - nth * A.pieces + (nth - int(quot(A.by_pieces, uint32_t(nth))) * A.pieces);
  piece -= piece >= A.pieces ? A.pieces : 0;
  n = A.n0 + nth;
  return true;
}

// Joins the pieces of a row that lie in LDS, `step` apart: four values from `dim` on, and
// log2 of the row's sum.  The sums are those that join_rows takes, in its order.
template <int D>
__device__ __forceinline__ float join_here(const float* at, int step, int pieces, int dim, f32x4& out) {
#pragma clang fp contract(off)
  constexpr int kAtOnce = 256 / D;
  float st[kWholePieces], M = -INFINITY;
#pragma unroll
  for (int p = 0; p < kWholePieces; ++p) {
    st[p] = p < pieces ? at[p * step + D + 2] : -INFINITY;
    M = fmaxf(M, st[p]);
  }
  const float base = M == -INFINITY ? 0.0f : M;
  float e[kWholePieces];
#pragma unroll
  for (int p = 0; p < kWholePieces; ++p) e[p] = fast_exp2(st[p] - base);
  static_assert(kWholePieces == 3, "the sum of eight lanes");
  const float L = (e[0] + e[2]) + e[1], by_L = L > 0.0f ? 1.0f / L : 0.0f;
  f32x4 sum[kAtOnce] = {};
#pragma unroll
  for (int p = 0; p < kWholePieces; ++p) {
    if (p >= pieces) break;
    const f32x4 x = *reinterpret_cast<const f32x4*>(at + p * step + dim);
    const float f = e[p] * by_L;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[p % kAtOnce][i] = __builtin_fmaf(x[i], f, sum[p % kAtOnce][i]);
  }
  out = sum[0] + sum[1];
  if constexpr (kAtOnce == 4) out = out + (sum[2] + sum[3]);
  return L > 0.0f ? base + fast_log2(L) : -INFINITY;
}

// WHOLE: a workgroup takes all pieces of a head, four waves each, and joins them itself.
template <int D, int MT, int GROUP, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(WHOLE ? kWholePieces * kThreads : kThreads, WHOLE ? 1 : 2) void k_attend_few(Args A) {
  static_assert(!WHOLE || MT == 1, "one row block");
  constexpr int kSteps = D / 32;        // matrix steps over the head dimension
  constexpr int kTiles = D / 16;        // 16-value tiles of the output
  constexpr int kVWords = D / 32;       // words of one key's values in a lane
  constexpr int kRowF = D + 4;          // floats of one merged row: sums, m, l
  constexpr int kPerTile = 32 / GROUP;  // look-ups of a tile
  extern __shared__ __align__(16) unsigned char lds_raw[];
  float* const lds = reinterpret_cast<float*>(lds_raw);
  __shared__ uint32_t none_all[kFewMaxChunk / 32];  // which look-ups of a tile found no page
  static_assert(kWholePieces * kFewChunk <= kFewMaxChunk, "the pieces' tiles side by side");

  const Paged& c = A.a.c;
  const int tid = WHOLE ? threadIdx.x % kThreads : threadIdx.x, lane = tid & 63, wave = tid >> 6;  // of the piece
  const int col = lane & 15, g = lane >> 4;
  int n, piece;
  if constexpr (WHOLE) {
    n = A.n0 + int(blockIdx.x);
    piece = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  } else if (!piece_of(A, n, piece)) {
    return;
  }
  const int b = int(quot(A.by_H, uint32_t(n))), h = n - b * c.H;

  const int2 mine = chunk_of(A.a.k, b);
  const int R = mine.y * A.a.G;
  if (R == 0 || R > kFewRows) return;
  const int len = paged_len(c, b);
  const int chunk = few_chunk(len);
  const int t0 = piece * chunk;
  if (!WHOLE && t0 >= len && piece > 0) return;
  const int left = len > t0 ? len - t0 : 0, keys = left < chunk ? left : chunk;  // of this piece
  const bool alone = len <= chunk;
  const int pieces = alone ? 1 : (len + chunk - 1) / chunk;
  const size_t place = WHOLE ? 0 : place_of(A, mine.x, b, h) + piece;   // of the first row
  // Rows of the look-ups, then the waves' sums.
  uint32_t* const where = reinterpret_cast<uint32_t*>(lds_raw) + (WHOLE ? piece * (kFewChunk / GROUP) : 0);
  uint32_t* const none_of = none_all + (WHOLE ? piece * (kFewChunk / 32) : 0);

  // Queries, on their way while the keys are looked up.
  u32x4 qf[MT][kSteps];
  int last[MT];  // last key of this piece that the row attends to
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = mt * 16 + col;
    const int i = int(quot(A.by_G, uint32_t(r)));
    last[mt] = r < R ? len - mine.y + i - t0 : -1;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      qf[mt][s] = u32x4{0, 0, 0, 0};
      if (r < R)
        qf[mt][s] = *reinterpret_cast<const u32x4*>(
            A.a.q.p + int64_t(mine.x + i) * A.a.q.ts + int64_t(h * A.a.G + r - i * A.a.G) * A.a.q.hs + s * 32 + g * 8);
    }
  }
  // Where the keys of this piece are.  A look-up that finds no page (or lies past
  // the end) points to row 0, whose bytes are dropped later.
  const int padded = (keys + 31) & ~31, lookups = padded / GROUP;
  for (int i = tid; i < ((lookups + 63) & ~63); i += kThreads) {
    uint32_t row = kNone;
    if (i * GROUP < keys) {
      const int64_t at = paged_row(c, b, h, t0 + i * GROUP);
      row = at < 0 ? kNone : uint32_t(at);
    }
    const uint64_t none = __ballot(row == kNone);
    if (i < lookups) {
      where[i] = row == kNone ? 0 : row;
      if (lane % kPerTile == 0) none_of[i / kPerTile] = uint32_t(none >> lane) & (0xffffffffu >> (32 - kPerTile));
    }
  }
  __syncthreads();

  // One tile of 32 keys as it is loaded.  K: this lane's keys are col of either half,
  // its values s*32 + g*8..; V: keys 4g..4g+3 of both halves, D/16 values of each.
  struct Tile {
    u32x4 k[2][kSteps];
    uint32_t v[8][kVWords];
  };
  auto fetch = [&](int tile, Tile& x) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key = tile + half * 16 + col;
      const uint16_t* at = c.k + (size_t(where[key / GROUP]) + key % GROUP) * D + g * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x.k[half][s] = load<STREAM, u32x4>(at + s * 32);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int key = tile + (i >> 2) * 16 + 4 * g + (i & 3);
      const uint16_t* at = c.v + (size_t(where[key / GROUP]) + key % GROUP) * D + col * (D / 16);
      if constexpr (kVWords == 4) {
        const u32x4 y = load<STREAM, u32x4>(at);
        x.v[i][0] = y.x, x.v[i][1] = y.y, x.v[i][2] = y.z, x.v[i][3] = y.w;
      } else {
        const u32x2 y = load<STREAM, u32x2>(at);
        x.v[i][0] = y.x, x.v[i][1] = y.y;
      }
    }
  };

  float nm[MT], l[MT];  // -m, sum of this lane's weights
  f32x4 acc[MT][kTiles];
  Loud loud{kSumLimit, 0.0f};
  float* const scores = A.scores ? first_score(A, mine.x, b, h, R) : nullptr;
  const int low = len - mine.y - t0;  // the first token's last key: all rows see the keys up to it
  const float by = A.a.c_log2;

  auto work = [&](int tile, Tile& x, bool checked) {
    float y[MT][8];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) a = mfma(x.k[half][s], qf[mt][s], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[mt][half * 4 + i] = a[i];
      }
    if (checked) {  // the same for the whole wave
      const uint32_t none = none_of[tile >> 5];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = (j >> 2) * 16 + 4 * g + (j & 3);
        const bool gone = (none >> (at / GROUP)) & 1;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (tile + at > last[mt] || gone) y[mt][j] = -INFINITY;
#pragma unroll
        for (int u = 0; u < kVWords; ++u)
          if (tile + at >= keys || gone) x.v[j][u] = 0;
      }
    }
    // For the sums of the weights, once the rows' sums are known.  These stores cost more
    // than their bytes: 4 rows of 131072 slots of 8 heads 24 us for 16.8 MB beside the 537 read.
    if (A.scores) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 16 + col;
        if (r < R) {
          float* to = scores + size_t(r) * A.score_stride + t0 + tile + 4 * g;
#pragma unroll
          for (int half = 0; half < 2; ++half)
            *reinterpret_cast<f32x4*>(to + half * 16) =
                f32x4{y[mt][half * 4] * by, y[mt][half * 4 + 1] * by, y[mt][half * 4 + 2] * by, y[mt][half * 4 + 3] * by};
        }
      }
    }
    u32x4 w[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float e[8], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = fast_exp2(__builtin_fmaf(y[mt][j], by, nm[mt]));
        sum += e[j];
      }
      if (__any(!(sum <= loud.limit))) {
        float top = y[mt][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, y[mt][j]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fminf(nm[mt], -top * by - loud.lift);
        const float f = fast_exp2(now - nm[mt]);
        nm[mt] = now;
        l[mt] *= f;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[mt][i] *= f;
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = fast_exp2(__builtin_fmaf(y[mt][j], by, now));
          sum += e[j];
        }
      }
      l[mt] += sum;
      w[mt] = u32x4{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])};
    }
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      const uint32_t pick = u & 1 ? 0x07060302u : 0x05040100u;  // the high or the low values of two words
      u32x4 vf;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vf[i] = __builtin_amdgcn_perm(x.v[2 * i + 1][u >> 1], x.v[2 * i][u >> 1], pick);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][u] = mfma(vf, w[mt], acc[mt][u]);
    }
  };
  for (bool again = false;; again = true) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      nm[mt] = kFar;
      l[mt] = 0.0f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) acc[mt][i] = f32x4{0, 0, 0, 0};
    }
    int first = wave;
    asm volatile("" : "+v"(first));          // or the first tile's addresses stay in registers
    for (int tile = first * 32; tile < keys; tile += kWaves * 32) {
      Tile cur;
      fetch(tile, cur);
      work(tile, cur, tile + 31 > low || none_of[tile >> 5] != 0);
    }
    float over = 0.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float here = 0.0f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) here += unless_finite(acc[mt][i].x, acc[mt][i].y, acc[mt][i].z, acc[mt][i].w);
      over += mt * 16 + col < R ? here : 0.0f;   // a place without a row weighs all keys alike
    }
    if (again || !__any(over != over)) break;
    loud = loud_of(4 * kFewMaxChunk / (32 * kWaves));   // four lanes a row and tile
  }

  // The waves' sums meet in LDS (over the look-ups), 16 rows at a time.
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
    l[mt] += __shfl_xor(l[mt], 16);
    l[mt] += __shfl_xor(l[mt], 32);
    const int r0 = mt * 16, rows_here = R - r0 < 16 ? R - r0 : 16;
    const int kept = WHOLE ? A.rows : 16;                 // rows that a wave leaves
    float* const of_piece = lds + (WHOLE ? piece * kWaves * kept * kRowF : 0);
    float* to = of_piece + (wave * kept + col) * kRowF;
    if (col < rows_here) {
#pragma unroll
      for (int r = 0; r < 4; ++r)  // values of row 4g + r of tile i: dim (4g + r) * kTiles + i
#pragma unroll
        for (int i = 0; i < kTiles; ++i) to[(4 * g + r) * kTiles + i] = acc[mt][i][r];
      if (g == 0) {
        to[D] = -nm[mt];
        to[D + 1] = l[mt];
      }
    }
    __syncthreads();
    for (int e = tid; e < rows_here * (D / 4); e += kThreads) {
      const int r = e / (D / 4), dim = e % (D / 4) * 4;
      float* at = of_piece + r * kRowF;
      float M = -kFar;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) M = fmaxf(M, at[w * kept * kRowF + D]);
      f32x4 sum = {0, 0, 0, 0};
      float L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* aw = at + w * kept * kRowF;
        const float f = fast_exp2(aw[D] - M);
        sum += *reinterpret_cast<const f32x4*>(aw + dim) * f;
        L = __builtin_fmaf(aw[D + 1], f, L);
      }
      const bool any = L > 0.0f;
      const float by_L = any ? 1.0f / L : 0.0f;
      sum *= by_L;
      if (any && unless_finite(sum.x, sum.y, sum.z, sum.w) != 0.0f) {   // each wave's share first
        sum = f32x4{0, 0, 0, 0};
        for (int w = 0; w < kWaves; ++w) {
          const float* aw = at + w * kept * kRowF;
          sum += *reinterpret_cast<const f32x4*>(aw + dim) * (fast_exp2(aw[D] - M) * by_L);
        }
      }
      sum = any ? sum : f32x4{0, 0, 0, 0};
      const float bsum = any ? M + fast_log2(L) : -INFINITY;
      if constexpr (WHOLE) {       // over the first wave's, which nobody else reads any more
        *reinterpret_cast<f32x4*>(at + dim) = sum;
        if (dim == 0) at[D + 2] = bsum;
        continue;
      }
      const size_t at_piece = place + (r0 + r) * pieces;
      if (A.scores && dim == 0) A.places.stat[at_piece] = bsum;
      if (alone) {
        const int i = int(quot(A.by_G, uint32_t(r0 + r)));
        finish(A, mine.x + i, h * A.a.G + r0 + r - i * A.a.G, dim, sum, bsum);
      } else {
        *reinterpret_cast<f32x4*>(A.places.part + at_piece * D + dim) = sum;
        if (dim == 0) A.places.stat[at_piece] = bsum;
      }
    }
  }
  if constexpr (WHOLE) {
    __shared__ float less[16];
    __syncthreads();
    const int threads = A.pieces * kThreads, step = kWaves * A.rows * kRowF;
    for (int e = threadIdx.x; e < R * (D / 4); e += threads) {
      const int r = e / (D / 4), dim = e % (D / 4) * 4;
      f32x4 out;
      const float bsum = join_here<D>(lds + r * kRowF, step, A.pieces, dim, out);
      const int i = int(quot(A.by_G, uint32_t(r)));
      finish(A, mine.x + i, h * A.a.G + r - i * A.a.G, dim, out, bsum);
      if (dim == 0) less[r] = -bsum == INFINITY ? -INFINITY : -bsum;
    }
    if (!A.scores) return;
    __syncthreads();
    for (int t = int(threadIdx.x) * 4; t < len; t += threads * 4) {
      float* to = c.weight + size_t(n) * c.room + t;
      float was[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) was[i] = t + i < len ? to[i] : 0.0f;
      weigh_four(A, scores, t, len, R, less, was, to);
    }
  }
}

// The sum of a row's pieces relative to 2^base, by N neighbouring lanes.
template <int N>
__device__ __forceinline__ float whole_sum(const float* st, int pieces, float& base) {
  const int lane = threadIdx.x % N;
  const float first = lane < pieces ? st[lane] : -INFINITY;  // the lane's first piece
  float M = first;
#pragma unroll 8
  for (int p = lane + N; p < pieces; p += N) M = fmaxf(M, st[p]);
#pragma unroll
  for (int off = N / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off));
  base = M == -INFINITY ? 0.0f : M;
  float L = fast_exp2(first - base);
#pragma unroll 8
  for (int p = lane + N; p < pieces; p += N) L += fast_exp2(st[p] - base);
#pragma unroll
  for (int off = N / 2; off > 0; off >>= 1) L += __shfl_xor(L, off);
  return L;
}

// Joins the pieces of a row, each weighted by its sum: D/4 lanes read one piece's
// outputs.  A row of at most kFewPieces of them is joined by a wave (256/D pieces at a
// time), one of more by the workgroup (1024/D at a time): the row's own count decides, so that
// its sums are taken in the same order in every call.  In a call where no head has more
// (SMALL) a workgroup takes a row a wave, otherwise one.
constexpr int kFewPieces = 8;
template <int D, bool SMALL>
__device__ __forceinline__ void join_rows(const Args& A, int n, int block, float* sums) {
  constexpr int kLanes = D / 4;
  const int b = int(quot(A.by_H, uint32_t(n))), h = n - b * A.a.c.H;
  const int2 mine = chunk_of(A.a.k, b);
  const int R = mine.y * A.a.G, r = SMALL ? block * kWaves + int(threadIdx.x >> 6) : block;
  const int len = paged_len(A.a.c, b), chunk = few_chunk(len);
  if (r >= R || R > kFewRows || len <= chunk) return;
  const int pieces = (len + chunk - 1) / chunk;
  const bool by_wave = SMALL || pieces <= kFewPieces;
  if (!SMALL && by_wave && threadIdx.x >= 64) return;
  const int at_once = (by_wave ? 64 : kThreads) / kLanes, thread = SMALL ? threadIdx.x % 64 : threadIdx.x;
  const int group = thread / kLanes, dim = thread % kLanes * 4;
  const size_t at = place_of(A, mine.x, b, h) + r * pieces;
  const float* st = A.places.stat + at;
  const float* part = A.places.part + at * D + dim;
  float base;
  const float L = by_wave ? whole_sum<kFewPieces>(st, pieces, base) : whole_sum<64>(st, pieces, base);
  const float by_L = L > 0.0f ? 1.0f / L : 0.0f;
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
  for (int p = group; p < pieces; p += at_once)
    sum += *reinterpret_cast<const f32x4*>(part + size_t(p) * D) * (fast_exp2(st[p] - base) * by_L);
  if (by_wave) {
#pragma unroll
    for (int off = kLanes; off < 64; off <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor(sum[i], off);
    if (group > 0) return;
  } else {
    *reinterpret_cast<f32x4*>(sums + group * D + dim) = sum;
    __syncthreads();
    if (group > 0) return;
    for (int i = 1; i < at_once; ++i) sum += *reinterpret_cast<const f32x4*>(sums + i * D + dim);
  }
  const int i = int(quot(A.by_G, uint32_t(r)));
  finish(A, mine.x + i, h * A.a.G + r - i * A.a.G, dim, sum, L > 0.0f ? base + fast_log2(L) : -INFINITY);
}

// What the slots of a piece receive from a sequence's few rows, four slots a thread.
__device__ __forceinline__ void weigh_piece(const Args& A, float* less) {
  int n, piece;
  if (!piece_of(A, n, piece)) return;
  const Paged& c = A.a.c;
  const int b = int(quot(A.by_H, uint32_t(n))), h = n - b * c.H;
  const int2 mine = chunk_of(A.a.k, b);
  const int R = mine.y * A.a.G, len = paged_len(c, b);
  const int chunk = few_chunk(len), t0 = piece * chunk, end = len - t0 < chunk ? len : t0 + chunk;
  if (R > kFewRows || t0 >= len) return;
  static_assert(kThreads == 8 * kFewRows, "eight lanes a row");
  const int pieces = (len + chunk - 1) / chunk, row = threadIdx.x >> 3;
  float* const to = c.weight + size_t(n) * c.room;
  float was[4];
  auto look = [&](int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) was[i] = t + i < end ? to[t + i] : 0.0f;
  };
  const int first = t0 + int(threadIdx.x) * 4;
  look(first);
  float base;
  const float L = whole_sum<8>(A.places.stat + place_of(A, mine.x, b, h) + row * pieces, row < R ? pieces : 0, base);
  if (threadIdx.x % 8 == 0) less[row] = L > 0.0f ? -(base + fast_log2(L)) : -INFINITY;   // a row that sees nothing gives nothing
  __syncthreads();
  const float* scores = first_score(A, mine.x, b, h, R);
  for (int t = first; t < end; t += kThreads * 4) {
    if (t > first) look(t);
    weigh_four(A, scores, t, end, R, less, was, to + t);
  }
}

// Both in one launch, as neither needs the other.  The workgroups that weigh are numbered
// as those that kept the scores, so that both lie on the same XCD, whose L2 may have them
// (80 sequences of 1100 slots, 4 heads each, 49.3 -> 46.5 us).
template <int D, bool SMALL>
__global__ __launch_bounds__(kThreads) void k_join_few(Args A, int joins, FastDiv by_joins) {
  __shared__ __align__(16) float lds[kThreads * 4];
  const int weighs = A.scores ? (A.units + 7) & ~7 : 0;
  if (int(blockIdx.x) < weighs) {
    weigh_piece(A, lds);
  } else {
    const uint32_t unit = blockIdx.x - weighs, nth = quot(by_joins, unit);
    join_rows<D, SMALL>(A, A.n0 + int(nth), int(unit - nth * by_joins.d), lds);
  }
}

template <int D, int MT, int GROUP, bool STREAM>
void attend_few(Args A, hipStream_t s) {
  const int heads = A.a.c.B * A.a.c.H;
  const bool small = A.pieces <= kFewPieces;
  const int joins = A.pieces == 1 ? 0 : (small ? (A.rows + kWaves - 1) / kWaves : A.rows);
  const FastDiv by_joins = fast_div(uint32_t(joins > 0 ? joins : 1));
  // At most 2^23 workgroups a launch (the grid counts work-items in 32 bits); a head has
  // 2^19 pieces and 32 joins at most.
  const int most = ((1 << 23) - 8) / (A.pieces + joins);
  const size_t keys = size_t(A.a.c.cap < kFewMaxChunk ? ((A.a.c.cap < kFewChunk ? kFewChunk : A.a.c.cap) + 127) & ~127 : kFewMaxChunk) / GROUP * 4;
  const size_t sums = size_t(kWaves) * 16 * (D + 4) * sizeof(float);
  for (A.n0 = 0; A.n0 < heads; A.n0 += most) {
    const int nh = heads - A.n0 < most ? heads - A.n0 : most;
    A.units = nh * A.pieces;
    k_attend_few<D, MT, GROUP, STREAM, false><<<unsigned(A.units), kThreads, keys > sums ? keys : sums, s>>>(A);
    const unsigned grid = unsigned(A.scores ? (A.units + 7) & ~7 : 0) + unsigned(nh) * unsigned(joins);
    if (grid == 0) continue;
    if (small) k_join_few<D, true><<<grid, kThreads, 0, s>>>(A, joins, by_joins);
    else k_join_few<D, false><<<grid, kThreads, 0, s>>>(A, joins, by_joins);
  }
}

template <int D, int GROUP, bool STREAM>
void attend_whole(Args A, hipStream_t s) {
  const int heads = A.a.c.B * A.a.c.H;
  const size_t keys = size_t(A.pieces) * kFewChunk / GROUP * 4;
  const size_t sums = size_t(A.pieces) * kWaves * A.rows * (D + 4) * sizeof(float);
  constexpr int kMost = 1 << 22;   // heads of a launch: below 2^32 work-items
  for (A.n0 = 0; A.n0 < heads; A.n0 += kMost) {
    const int nh = heads - A.n0 < kMost ? heads - A.n0 : kMost;
    k_attend_few<D, 1, GROUP, STREAM, true>
        <<<unsigned(nh), unsigned(A.pieces) * kThreads, keys > sums ? keys : sums, s>>>(A);
  }
}

// Whether a workgroup takes all pieces of a head, or one (the results are the same
// bits).  It saves the second launch and the pieces' way through memory, but one that
// takes several fills a CU: 100 heads or fewer leave CUs without work, and so does a last
// round of them.  Heads of 1100 slots, 7 rows, us (one launch : two): 64 heads 16.9 : 13.3,
// 96 heads 17.3 : 18.9, 256 heads 27.4 : 30.8 (with weights 33.1 : 39.6), 288 heads 46.4 :
// 36.3, 512 heads 53.5 : 56.1, 2048 heads 207 : 228 (with weights the same); 400 slots with
// weights, 256 heads 16.5 : 19.0.  The host knows no lengths: `pieces` are those of the
// longest one that the table, or max_len, has room for.  256 heads of about 1090 slots, 7 rows, in
// tables of 1536, 2048, 4096, 32768 slots: 27, 35, 38, 45 us, with weights 33, 43, 47, 64; with
// max_len 1536 27 and 33 in all of them.
bool whole_heads(int heads, int pieces, int rows, bool weights) {
  if (rows > 16 || pieces > kWholePieces) return false;
  if (pieces == 1) return weights;
  constexpr int kCUs = 256;
  const int64_t rounds = (int64_t(heads) + kCUs - 1) / kCUs;
  return heads >= 96 && (rounds == 1 || heads * int64_t(8) >= rounds * kCUs * 7);
}

template <int D>
void attend_rows(const Args& A, hipStream_t s) {
  const bool fours = A.a.c.bs % 4 == 0;
  // Keys and values out of pools that are a good part of the last-level cache (256 MB)
  // are read past the caches, which they would only empty: 89 us against 101 on one
  // sequence of 131072 slots (537 MB), 40.3 against 42.6 on 64 sequences of 1100 that the
  // cache does not hold yet (145 MB; found there again by the next call, 39 against 34).
  // 17 to 32 rows of 128 values: out of pools past it, 95 against 107 (537 MB), 134 against
  // 147 with weights and 103 against 100 without (436 MB); 41 against 37 (145 MB).  Of 64
  // values never: 57 against 48 (218 MB), 285 against 282 (805 MB).
  const uint64_t pools = uint64_t(A.a.c.n_blocks) * A.a.c.H * A.a.c.bs * D * 4;
  const bool stream = pools > (uint64_t(A.rows <= 16 ? 96 : 256) << 20);
  if (whole_heads(A.a.c.B * A.a.c.H, A.pieces, A.rows, A.scores != nullptr)) {
    if (fours && stream) attend_whole<D, 4, true>(A, s);
    else if (fours) attend_whole<D, 4, false>(A, s);
    else attend_whole<D, 1, false>(A, s);
  } else if (A.rows <= 16) {
    if (fours && stream) attend_few<D, 1, 4, true>(A, s);
    else if (fours) attend_few<D, 1, 4, false>(A, s);
    else attend_few<D, 1, 1, false>(A, s);
  } else {
    // One row block of 32, not two of 16 that read each key twice: 99.6 us against 107 (13
    // sequences of 8192 slots, d 128), 36.8 against 35.6 (64 of 1100).
    if (D == 128 && fours && stream) attend_few<128, 2, 4, true>(A, s);
    else if (fours) attend_few<D, 2, 4, false>(A, s);
    else attend_few<D, 2, 1, false>(A, s);
  }
}

}  // namespace

AttendWs attend_ws(const Paged& c, const Chunks& k, int G) {
  AttendWs w{};
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = (off + n + 63) & ~size_t(63);
    return at;
  };
  w.few_rows = int64_t(G) * k.max_new < kFewRows ? G * k.max_new : kFewRows;
  w.few_pieces = few_max_pieces(c.cap);
  const bool many = int64_t(G) * k.max_new > kFewRows;
  const int most = tile_max_pieces(c.cap), few = w.few_rows * w.few_pieces;
  w.slots = many ? first_slot(k.n_tokens, c.B, G, most) + 1 : 0;
  w.places.most = many && most > w.few_pieces ? most : w.few_pieces;
  w.places.each = many && kTileWork * kTileRows > few ? kTileWork * kTileRows : few;
  w.places.total = first_place(w.places, k.n_tokens, c.B, G);
  const size_t n = size_t(w.places.total) * c.H;
  w.part = take(w.places.most > 1 ? n * c.D : 0);
  w.stat = take(w.places.most > 1 || c.weight ? n : 0);
  w.score_stride = (c.cap + 31) & ~31;
  w.scores = take(c.weight ? size_t(score_rows(k.n_tokens, c.B, G, w.few_rows)) * c.H * w.score_stride : 0);
  w.lse = take(c.weight ? size_t(k.n_tokens) * G * c.H : 0);
  w.total = off;
  return w;
}

hipError_t launch_paged_attend(const AttendCall& a, float* ws, hipStream_t s) {
  const AttendWs w = attend_ws(a.c, a.k, a.G);
  Args A{};
  A.a = a;
  if (a.c.weight && !a.lse) A.a.lse = ws + w.lse;
  A.pieces = w.few_pieces;
  A.rows = w.few_rows;
  A.by_G = fast_div(uint32_t(a.G));
  A.by_pieces = fast_div(uint32_t(A.pieces));
  A.by_H = fast_div(uint32_t(a.c.H));
  A.places = w.places;
  A.places.part = ws + w.part;
  A.places.stat = ws + w.stat;
  A.scores = a.c.weight ? ws + w.scores : nullptr;
  A.score_stride = w.score_stride;
  if (a.c.D == 128) attend_rows<128>(A, s);
  else attend_rows<64>(A, s);
  if (w.slots > 0) {
    AttendCall t = a;
    t.lse = A.a.lse;
    const hipError_t e = launch_attend_tiles(t, A.places, w.slots, s);
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace kvc
