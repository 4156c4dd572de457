// Storing, loading and appending rows of the 8-bit paged cache on gfx950.
//
// A page of one head is bs x D codes under one fp32 scale.  Storing needs the
// largest magnitude of the page before the first code can be written: the page
// stays in registers between the two (one wave for small pages, a workgroup
// for larger ones), so every row is read once; only pages past what a
// workgroup holds are read twice.  All three are bound by HBM: 1792 heads' 256
// kept rows of 768 are stored in 70 us (5.0 TB/s), a 16384-row cache of 32 heads
// in 61 (5.8 TB/s).
//
// The arithmetic is one rounding at a time (this unit is compiled without
// contraction): e4m3 scales are powers of two, so x / scale is exact and the
// code is the one rounding; int8 rounds 1 / scale and the product, then the
// code.
#include "kvc_q8.h"

namespace kvc {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

struct Scale {
  float scale, inv;
};

// The scale of a page whose largest magnitude is amax (bf16 bits).
template <int FMT>
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
  const uint32_t f = amax_bits << 16;
  if constexpr (FMT == KVC_Q8_E4M3) {
    // amax = m * 2^k, 448 = 1.75 * 2^8: e = k - 8, one more when m > 1.75.
    int e = int(f >> 23) - 127 - 8 + ((f & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -126 ? -126 : e;
    return Scale{__uint_as_float(uint32_t(e + 127) << 23), __uint_as_float(uint32_t(127 - e) << 23)};
  } else {
    const float s = fmaxf(__uint_as_float(f) / 127.0f, 0x1p-126f);
    return Scale{s, 1.0f / s};
  }
}

// Four codes of four values (already divided by the scale).
template <int FMT>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  if constexpr (FMT == KVC_Q8_E4M3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
  } else {
    // adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and
    // leaves it in the low byte
    const float r = 12582912.0f;
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b + r), __float_as_uint(a + r), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d + r), __float_as_uint(c + r), 0x04000c0cu);
    return lo | hi;
  }
}

template <int FMT>
__device__ __forceinline__ void value4(uint32_t w, float* x) {
  if constexpr (FMT == KVC_Q8_E4M3) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = float(int8_t(w >> (8 * i)));
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight bf16 values (as loaded) to eight codes.
template <int FMT>
__device__ __forceinline__ u32x2 code8(u32x4 x, float inv) {
  return u32x2{code4<FMT>(lo_f32(x.x) * inv, hi_f32(x.x) * inv, lo_f32(x.y) * inv, hi_f32(x.y) * inv),
               code4<FMT>(lo_f32(x.z) * inv, hi_f32(x.z) * inv, lo_f32(x.w) * inv, hi_f32(x.w) * inv)};
}

// Largest magnitudes of two halves at a time: bf16 magnitudes order like
// their bits.
__device__ __forceinline__ u16x2 amax2(u16x2 m, uint32_t w) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w & 0x7fff7fffu));
}
__device__ __forceinline__ u16x2 amax8(u16x2 m, u32x4 x) {
  return amax2(amax2(amax2(amax2(m, x.x), x.y), x.z), x.w);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t y = uint32_t(__shfl_xor(int(x), off));
    x = x > y ? x : y;
  }
  return x;
}

// One (head, page, K or V) per unit of WAVES waves.  PIECES > 0: each lane
// holds that many 16-value pieces of the page; 0: the page is read twice.
template <int D, int FMT, int WAVES, int PIECES>
__global__ __launch_bounds__(kThreads) void k_q8_store(Q8 c, int T, int TS,
                                                       const int32_t* __restrict__ kept, int n_kept,
                                                       const u32x4* __restrict__ k,
                                                       const u32x4* __restrict__ v, int pages,
                                                       uint32_t u0, uint32_t units) {
  constexpr int kLanes = WAVES * 64, kRowPieces = D / 16;
  __shared__ uint32_t wave_top[4];
  const uint32_t u = u0 + blockIdx.x * (4 / WAVES) + (WAVES == 1 ? threadIdx.x >> 6 : 0);
  if (u >= units) return;
  const int lane = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t kv = u & 1, pg = (u >> 1) % uint32_t(pages), n = (u >> 1) / uint32_t(pages);
  const int b = n / c.H, h = n % c.H;
  const int top = kept ? n_kept : T;
  int L = q8_len(c, b);
  L = L < top ? L : top;
  const int s0 = int(pg) * c.bs;
  if (s0 >= L) return;  // the same for the whole unit
  const int page = q8_page(c, b, pg);
  if (page < 0) return;
  const int rows = L - s0 < c.bs ? L - s0 : c.bs;
  const u32x4* src = (kv ? v : k) + size_t(n) * TS * (D / 8);
  const int32_t* kn = kept ? kept + size_t(n) * n_kept + s0 : nullptr;
  const int total = rows * kRowPieces;
  auto read = [&](int i, u32x4& a, u32x4& z) {
    const int r = i / kRowPieces, p = i % kRowPieces;
    const int t = kn ? kn[r] : T - L + s0 + r;
    a = z = u32x4{0, 0, 0, 0};
    if (t >= 0 && t < T) {
      const u32x4* at = src + size_t(t) * (D / 8) + p * 2;
      a = __builtin_nontemporal_load(at);
      z = __builtin_nontemporal_load(at + 1);
    }
  };
  u16x2 m = {0, 0};
  u32x4 x[PIECES > 0 ? PIECES : 1][2];
  if constexpr (PIECES > 0) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int e = lane + i * kLanes;
      x[i][0] = x[i][1] = u32x4{0, 0, 0, 0};
      if (e < total) read(e, x[i][0], x[i][1]);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) m = amax8(amax8(m, x[i][0]), x[i][1]);
  } else {
    for (int e = lane; e < total; e += kLanes) {
      read(e, x[0][0], x[0][1]);
      m = amax8(amax8(m, x[0][0]), x[0][1]);
    }
  }
  uint32_t amax = wave_max(m.x > m.y ? m.x : m.y);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = amax;
    __syncthreads();
    const uint32_t a = wave_top[0] > wave_top[1] ? wave_top[0] : wave_top[1];
    const uint32_t z = wave_top[2] > wave_top[3] ? wave_top[2] : wave_top[3];
    amax = a > z ? a : z;
  }
  const Scale sc = scale_of<FMT>(amax);
  const size_t ph = size_t(page) * c.H + h;
  if (lane == 0) (kv ? c.vs : c.ks)[ph] = sc.scale;
  u32x4* dst = reinterpret_cast<u32x4*>((kv ? c.v : c.k) + ph * c.bs * D);
  if constexpr (PIECES > 0) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int e = lane + i * kLanes;
      if (e < total) {
        const u32x2 a = code8<FMT>(x[i][0], sc.inv), z = code8<FMT>(x[i][1], sc.inv);
        dst[e] = u32x4{a.x, a.y, z.x, z.y};
      }
    }
  } else {
    for (int e = lane; e < total; e += kLanes) {
      read(e, x[0][0], x[0][1]);
      const u32x2 a = code8<FMT>(x[0][0], sc.inv), z = code8<FMT>(x[0][1], sc.inv);
      dst[e] = u32x4{a.x, a.y, z.x, z.y};
    }
  }
}

// Values code * scale as bf16 rows: 8 values of K and of V per thread, so that a
// wave's stores are whole lines (with 16 values a thread, two stores 32 bytes
// apart, it ran at 3.5 TB/s against 5.7 on the 16K and Qwen-shaped caches;
// two or four rows a thread were 4 and 8 % slower than one).
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_q8_load(Q8 c, int T, int TS, int chunks,
                                                      u32x4* __restrict__ k_out,
                                                      u32x4* __restrict__ v_out, int h0) {
  constexpr int kRowPieces = D / 8, kRows = kThreads / kRowPieces;
  const int n = h0 + int(blockIdx.x / unsigned(chunks));
  const int r = int(blockIdx.x % unsigned(chunks)) * kRows + int(threadIdx.x) / kRowPieces;
  const int p = int(threadIdx.x) % kRowPieces;
  if (r >= T) return;
  const int b = n / c.H, h = n % c.H;
  const int L = q8_len(c, b);
  const int64_t j = int64_t(r) - T + L;  // position of this row
  u32x2 x[2] = {{0, 0}, {0, 0}};
  float s[2] = {0.f, 0.f};
  if (j >= 0) {
    const uint32_t jb = quot(c.div, uint32_t(j));
    const int page = q8_page(c, b, int(jb));
    if (page >= 0) {
      const size_t ph = size_t(page) * c.H + h;
      const size_t at = (ph * c.bs + (uint32_t(j) - jb * c.div.d)) * kRowPieces + p;
      if (k_out) {
        x[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c.k) + at);
        s[0] = c.ks[ph];
      }
      if (v_out) {
        x[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c.v) + at);
        s[1] = c.vs[ph];
      }
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    u32x4* out = kv ? v_out : k_out;
    if (!out) continue;
    u32x4 w;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float f[4];
      value4<FMT>(x[kv][g], f);
      w[2 * g] = pack_bf16(f[0] * s[kv], f[1] * s[kv]);
      w[2 * g + 1] = pack_bf16(f[2] * s[kv], f[3] * s[kv]);
    }
    __builtin_nontemporal_store(w, out + (size_t(n) * TS + r) * kRowPieces + p);
  }
}

// One wave per (head, touched page), for K and V at once: it waits for memory
// three times (length, table, scale), and fewer waves wait fewer times (14 us for
// 9472 heads with a wave for each of K and V, 10 so).  The first 128 pieces
// of the new rows (8 rows at D = 128) are on their way while the page is looked
// up, and stay in registers until they are coded; what is past them is read
// twice.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_q8_append(Q8 c, int W,
                                                        const int32_t* __restrict__ n_new,
                                                        const u32x4* __restrict__ k_new,
                                                        const u32x4* __restrict__ v_new, int pages,
                                                        uint32_t u0, uint32_t units) {
  constexpr int kRowPieces = D / 8;  // of the new rows; of the codes: D / 16
  const uint32_t u = u0 + blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= units) return;
  const int lane = threadIdx.x & 63;
  const uint32_t pi = u % uint32_t(pages), n = u / uint32_t(pages);
  const int b = n / c.H, h = n % c.H;
  const int L = q8_len(c, b);
  int mine = W;  // rows this sequence appends
  if (n_new) {
    mine = n_new[b];
    mine = mine < 0 ? 0 : (mine < W ? mine : W);
    if (mine == 0) return;
  }
  const int first = L > mine ? L - mine : 0;  // first new position that exists
  const int pg = int(quot(c.div, uint32_t(first))) + int(pi);
  const int s0 = pg * c.bs;
  if (s0 >= L) return;
  const int a = first > s0 ? first - s0 : 0;              // first new slot
  const int e = L - s0 < c.bs ? L - s0 : c.bs;            // past the last one
  const size_t from = (size_t(n) * W + (s0 + a - (L - W))) * kRowPieces;
  const u32x4* src[2] = {k_new + from, v_new + from};
  const int total = (e - a) * kRowPieces;
  u32x4 x[2][2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[kv][j] = u32x4{0, 0, 0, 0};
      if (lane + 64 * j < total) x[kv][j] = src[kv][lane + 64 * j];
    }
  const int page = q8_page(c, b, pg);
  if (page < 0) return;
  const size_t ph = size_t(page) * c.H + h;
  float* scale[2] = {c.ks + ph, c.vs + ph};
  float old[2] = {0.0f, 0.0f};
  if (a > 0) old[0] = *scale[0], old[1] = *scale[1];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* codes = (kv ? c.v : c.k) + ph * c.bs * D;
    u16x2 m = amax8(amax8(u16x2{0, 0}, x[kv][0]), x[kv][1]);
    for (int i = lane + 128; i < total; i += 64) m = amax8(m, src[kv][i]);
    Scale sc = scale_of<FMT>(wave_max(m.x > m.y ? m.x : m.y));
    if (a > 0) {
      if (old[kv] >= sc.scale) {
        sc.scale = old[kv];
        sc.inv = 1.0f / old[kv];
      } else {
        // earlier rows again under the larger scale
        const float ratio = FMT == KVC_Q8_E4M3 ? old[kv] / sc.scale : old[kv] * sc.inv;
        u32x4* rows = reinterpret_cast<u32x4*>(codes);
        for (int i = lane; i < a * (D / 16); i += 64) {
          u32x4 w = rows[i];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float f[4];
            value4<FMT>(w[g], f);
            w[g] = code4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
          }
          rows[i] = w;
        }
      }
    }
    if (lane == 0 && (a == 0 || sc.scale != old[kv])) *scale[kv] = sc.scale;
    u32x2* dst = reinterpret_cast<u32x2*>(codes + size_t(a) * D);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (lane + 64 * j < total) dst[lane + 64 * j] = code8<FMT>(x[kv][j], sc.inv);
    for (int i = lane + 128; i < total; i += 64) dst[i] = code8<FMT>(src[kv][i], sc.inv);
  }
}

// Units in launches of at most 2^23 workgroups (the grid counts work-items in
// 32 bits).
template <class F>
void in_launches(uint64_t units, uint32_t per_block, F launch) {
  const uint64_t step = uint64_t(1) << 23;
  for (uint64_t u0 = 0; u0 < units; u0 += step * per_block) {
    const uint64_t left = units - u0;
    const uint64_t blocks = (left + per_block - 1) / per_block;
    launch(uint32_t(u0), unsigned(blocks < step ? blocks : step));
  }
}

template <int D, int FMT>
void store(const Q8& c, int T, int TS, const int32_t* kept, int n_kept, const u32x4* k,
           const u32x4* v, hipStream_t s) {
  const int top0 = kept ? n_kept : T, top = top0 < c.cap ? top0 : c.cap;
  const int pages = (top + c.bs - 1) / c.bs;
  const uint64_t units = uint64_t(c.B) * c.H * pages * 2;
  const int pieces = c.bs * (D / 16);
#define KVC_STORE(WAVES, PIECES)                                                                \
  in_launches(units, 4 / WAVES, [&](uint32_t u0, unsigned blocks) {                             \
    k_q8_store<D, FMT, WAVES, PIECES><<<blocks, kThreads, 0, s>>>(c, T, TS, kept, n_kept, k, v, \
                                                                  pages, u0, uint32_t(units)); \
  })
  if (pieces <= 64) KVC_STORE(1, 1);
  else if (pieces <= 128) KVC_STORE(1, 2);
  else if (pieces <= 256) KVC_STORE(4, 1);
  else if (pieces <= 512) KVC_STORE(4, 2);
  else if (pieces <= 1024) KVC_STORE(4, 4);
  else KVC_STORE(4, 0);
#undef KVC_STORE
}

template <int D, int FMT>
void append(const Q8& c, int W, const int32_t* n_new, const u32x4* k, const u32x4* v,
            hipStream_t s) {
  int pages = (W + c.bs - 2) / c.bs + 1;  // pages that W positions can touch
  pages = pages < c.tb ? pages : c.tb;
  const uint64_t units = uint64_t(c.B) * c.H * pages;
  in_launches(units, 4, [&](uint32_t u0, unsigned blocks) {
    k_q8_append<D, FMT><<<blocks, kThreads, 0, s>>>(c, W, n_new, k, v, pages, u0, uint32_t(units));
  });
}

template <int D, int FMT>
void load(const Q8& c, int T, int TS, u32x4* k, u32x4* v, hipStream_t s) {
  const int rows = kThreads / (D / 8);
  const int chunks = (T + rows - 1) / rows;
  const int heads = c.B * c.H;
  const int per = (1 << 23) / chunks > 0 ? (1 << 23) / chunks : 1;
  for (int h0 = 0; h0 < heads; h0 += per) {
    const int nh = heads - h0 < per ? heads - h0 : per;
    k_q8_load<D, FMT><<<unsigned(nh) * unsigned(chunks), kThreads, 0, s>>>(c, T, TS, chunks, k, v, h0);
  }
}

}  // namespace

#define KVC_Q8_CASES(CALL)                                                     \
  if (c.D == 128 && c.fmt == KVC_Q8_E4M3) CALL(128, KVC_Q8_E4M3);              \
  else if (c.D == 128) CALL(128, KVC_Q8_INT8);                                 \
  else if (c.fmt == KVC_Q8_E4M3) CALL(64, KVC_Q8_E4M3);                        \
  else CALL(64, KVC_Q8_INT8)

hipError_t launch_q8_store(const Q8& c, int T, int TS, const int32_t* kept, int n_kept,
                           const void* k, const void* v, hipStream_t s) {
  const u32x4* kk = static_cast<const u32x4*>(k);
  const u32x4* vv = static_cast<const u32x4*>(v);
#define CALL(D, F) store<D, F>(c, T, TS, kept, n_kept, kk, vv, s)
  KVC_Q8_CASES(CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_q8_load(const Q8& c, int T, int TS, void* k_out, void* v_out, hipStream_t s) {
  u32x4* kk = static_cast<u32x4*>(k_out);
  u32x4* vv = static_cast<u32x4*>(v_out);
#define CALL(D, F) load<D, F>(c, T, TS, kk, vv, s)
  KVC_Q8_CASES(CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_q8_append(const Q8& c, int W, const int32_t* n_new, const void* k_new,
                            const void* v_new, hipStream_t s) {
  const u32x4* kk = static_cast<const u32x4*>(k_new);
  const u32x4* vv = static_cast<const u32x4*>(v_new);
#define CALL(D, F) append<D, F>(c, W, n_new, kk, vv, s)
  KVC_Q8_CASES(CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace kvc
