// Rotary positions of new tokens, alone or on the way into a bf16 paged cache.
//
// A pair (x0, x1) of a row turns by a = position * freq[i].  The angle is formed in
// turns, position * (freq / 2 pi), in fp64 and reduced there: at position 131072 an
// fp32 product would be off by 2^-8 of a radian.  Cosines and sines of a
// token are taken once, into LDS, and serve all its heads (Llama-shaped: 64 angles for
// 40 rows of 128 values).  What remains is a copy: 2 * d bytes in, 2 * d out a row.
//
// Every rotated value is read and written by the one thread that has its pair, so y
// may be x.  A thread takes eight pairs, 16 bytes of either half of the rotated part (of
// any alignment: its second half starts anywhere), or four interleaved pairs, which are 16
// neighbouring bytes.
//
// Measured: 16384 tokens of 32 heads of 128, 38.8 us (134 MB in, 134 out: 6.9 TB/s, part of
// it out of the last-level cache).  A token a workgroup leaves the few tokens of a decode
// step to the latency of angles and rows, and an append to that of start -> length -> table ->
// rows: 64 tokens of 36 heads 4.1 us.
#include "kvc_paged.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) Loose { u32x4 x; };  // 16 bytes at any row offset

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;   // head_dim / 2

struct Turns {
  float c[kMaxPairs], s[kMaxPairs];
};

__device__ __forceinline__ void turn_of(const RopePlan& f, int at, int i, float& c, float& s) {
  const double turns = double(at) * (f.freq[i] * 0.15915494309189535);  // 1 / 2 pi
  const float part = float(turns - rint(turns));
  float si, co;
  sincospif(2.0f * part, &si, &co);
  c = co * f.mscale;
  s = si * f.mscale * f.sign;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Items of a row that rotates: eight pairs each (four when interleaved), then the copied
// values by eight.
struct Shape {
  int r, half, turn_items, items;
};
__host__ __device__ inline Shape shape_of(const RopePlan& f, int D) {
  Shape s;
  s.r = f.r;
  s.half = f.r / 2;
  s.turn_items = f.interleaved ? (f.r + 7) / 8 : (s.half + 7) / 8;
  const int from = f.interleaved ? s.turn_items * 8 : f.r;  // the last interleaved piece carries its copies
  s.items = s.turn_items + (D - from + 7) / 8;
  return s;
}

__device__ __forceinline__ void row_item(const RopePlan& f, const Shape& sh, const Turns& t, int D,
                                         int item, const uint16_t* x, uint16_t* y) {
  if (item < sh.turn_items && f.interleaved) {
    u32x4 a = *reinterpret_cast<const u32x4*>(x + item * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = item * 4 + j;
      if (i < sh.half) {
        const float x0 = lo_f(a[j]), x1 = hi_f(a[j]), c = t.c[i], s = t.s[i];
        a[j] = pack_bf16(x0 * c - x1 * s, x1 * c + x0 * s);
      }
    }
    *reinterpret_cast<u32x4*>(y + item * 8) = a;
  } else if (item < sh.turn_items) {
    const int i0 = item * 8, n = sh.half - i0 < 8 ? sh.half - i0 : 8;
    if (n == 8) {
      u32x4 a = reinterpret_cast<const Loose*>(x + i0)->x;
      u32x4 b = reinterpret_cast<const Loose*>(x + sh.half + i0)->x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a0 = lo_f(a[j]), a1 = hi_f(a[j]), b0 = lo_f(b[j]), b1 = hi_f(b[j]);
        const float c0 = t.c[i0 + 2 * j], c1 = t.c[i0 + 2 * j + 1];
        const float s0 = t.s[i0 + 2 * j], s1 = t.s[i0 + 2 * j + 1];
        a[j] = pack_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
        b[j] = pack_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
      }
      reinterpret_cast<Loose*>(y + i0)->x = a;
      reinterpret_cast<Loose*>(y + sh.half + i0)->x = b;
    } else {
      for (int j = 0; j < n; ++j) {
        const float x0 = lo_f(x[i0 + j]), x1 = lo_f(x[sh.half + i0 + j]);
        const float c = t.c[i0 + j], s = t.s[i0 + j];
        y[i0 + j] = to_bf16(x0 * c - x1 * s);
        y[sh.half + i0 + j] = to_bf16(x1 * c + x0 * s);
      }
    }
  } else if (x != y) {
    const int i0 = (f.interleaved ? sh.turn_items * 8 : sh.r) + (item - sh.turn_items) * 8;
    const int n = D - i0 < 8 ? D - i0 : 8;
    if (n == 8) {
      reinterpret_cast<Loose*>(y + i0)->x = reinterpret_cast<const Loose*>(x + i0)->x;
    } else {
      for (int j = 0; j < n; ++j) y[i0 + j] = x[i0 + j];
    }
  }
}

// One token a workgroup.
__global__ __launch_bounds__(kThreads) void k_rope(RopePlan f, int heads, int D, FastDiv by_items,
                                                   const int32_t* positions, Rows x, Rows y) {
  __shared__ Turns t;
  const int token = blockIdx.x;
  const Shape sh = shape_of(f, D);
  if (threadIdx.x < sh.half)
    turn_of(f, positions[token], threadIdx.x, t.c[threadIdx.x], t.s[threadIdx.x]);
  __syncthreads();
  const uint16_t* xt = x.p + token * x.ts;
  uint16_t* yt = y.p + token * y.ts;
  for (uint32_t i = threadIdx.x; i < uint32_t(heads) * sh.items; i += kThreads) {
    const uint32_t h = quot(by_items, i);
    row_item(f, sh, t, D, int(i - h * sh.items), xt + h * x.hs, yt + h * y.hs);
  }
}

// One token a workgroup: its query heads, then its key heads, then its values, so that
// the angles serve both and one launch does for a step (64 tokens of 28 query and 4 KV heads
// of 128 4.1 us, 981 tokens of 32 and 8 of 64 6.0: latency).
__global__ __launch_bounds__(kThreads) void k_paged_append(
    Paged c, Chunks k, const int32_t* positions, RopePlan f, int q_heads, FastDiv by_items,
    Rows q, Rows q_out, Rows k_new, Rows v_new) {
  __shared__ Turns t;
  const int token = blockIdx.x, D = c.D;
  const int b = last_at_or_below(k, token, [](int s, int) { return s; });
  const int2 mine = chunk_of(k, b);
  const int i_new = token - mine.x;
  if (i_new < 0 || i_new >= mine.y) return;
  const int slot = paged_len(c, b) - mine.y + i_new;
  const int at = positions ? positions[token] : slot;
  const Shape sh = shape_of(f, D);
  if (threadIdx.x < sh.half) turn_of(f, at, threadIdx.x, t.c[threadIdx.x], t.s[threadIdx.x]);
  __syncthreads();
  int64_t row = -1;
  if (slot >= 0) row = paged_row(c, b, 0, slot);
  const uint32_t n_q = uint32_t(q_heads) * sh.items;
  const uint32_t n_k = row < 0 ? 0 : uint32_t(c.H) * sh.items;
  const uint32_t n_v = row < 0 ? 0 : uint32_t(c.H) * (D / 8);
  for (uint32_t i = threadIdx.x; i < n_q + n_k + n_v; i += kThreads) {
    if (i < n_q) {
      const uint32_t h = quot(by_items, i);
      row_item(f, sh, t, D, int(i - h * sh.items), q.p + token * q.ts + h * q.hs,
               q_out.p + token * q_out.ts + h * q_out.hs);
    } else if (i < n_q + n_k) {
      const uint32_t h = quot(by_items, i - n_q);
      row_item(f, sh, t, D, int(i - n_q - h * sh.items), k_new.p + token * k_new.ts + h * k_new.hs,
               c.k + (row + int64_t(h) * c.bs) * D);
    } else {
      const uint32_t e = i - n_q - n_k, h = e / (D / 8), p = e % (D / 8);
      *reinterpret_cast<u32x4*>(c.v + (row + int64_t(h) * c.bs) * D + p * 8) =
          *reinterpret_cast<const u32x4*>(v_new.p + token * v_new.ts + h * v_new.hs + p * 8);
    }
  }
  if (c.weight && row >= 0) {
    for (int h = threadIdx.x; h < c.H; h += kThreads) {
      const size_t at_slot = (size_t(b) * c.H + h) * c.room + slot;
      c.weight[at_slot] = 0.0f;
      c.pos[at_slot] = at;
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopePlan& f, int n_tokens, int heads, int D, const int32_t* positions,
                       const Rows& x, const Rows& y, hipStream_t s) {
  const FastDiv by_items = fast_div(uint32_t(shape_of(f, D).items));
  k_rope<<<unsigned(n_tokens), kThreads, 0, s>>>(f, heads, D, by_items, positions, x, y);
  return hipGetLastError();
}

hipError_t launch_paged_append(const Paged& c, const Chunks& k, const int32_t* positions,
                               const RopePlan& f, int q_heads, const Rows& q, const Rows& q_out,
                               const Rows& k_new, const Rows& v_new, hipStream_t s) {
  const FastDiv by_items = fast_div(uint32_t(shape_of(f, c.D).items));
  k_paged_append<<<unsigned(k.n_tokens), kThreads, 0, s>>>(c, k, positions, f, q_heads, by_items, q,
                                                           q_out, k_new, v_new);
  return hipGetLastError();
}

}  // namespace kvc
