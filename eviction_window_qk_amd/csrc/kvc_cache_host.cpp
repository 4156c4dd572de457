// Host side of the 8-bit paged cache and of the page tables: validates every
// argument of their C entry points and enqueues the kernels.  No allocation on
// the device, no synchronisation, no global state.
#include <math.h>

#include <algorithm>
#include <new>

#include "kvc_host.h"
#include "kvc_pages.h"
#include "kvc_q8.h"

namespace kvc {
namespace {

// Makes the device of `stream` current for the launches of a call.  The implicit
// streams are the current device's already, and their handles no objects that the
// runtime could be asked about.
struct OnDeviceOf {
  int was = -1;
  bool ok = true;
  explicit OnDeviceOf(hipStream_t stream) {
    if (stream == nullptr || stream == hipStreamPerThread) return;
    int cur = -1, dev = -1;
    ok = hipGetDevice(&cur) == hipSuccess && hipStreamGetDevice(stream, &dev) == hipSuccess;
    if (ok && cur != dev) {
      ok = hipSetDevice(dev) == hipSuccess;
      was = cur;
    }
  }
  ~OnDeviceOf() {
    if (was >= 0) (void)hipSetDevice(was);
  }
};

template <class F>
int launch_on(void* stream, F launch) {
  const hipStream_t s = hipStream_t(stream) == hipStreamLegacy ? nullptr : hipStream_t(stream);
  OnDeviceOf dev(s);
  return dev.ok ? launch_status(launch(s)) : KVC_EDEVICE;
}

size_t pool_bytes(const kvc_q8_cache* c) {
  return size_t(c->n_blocks) * c->kv_heads * c->block_size * c->head_dim;
}
size_t scale_bytes(const kvc_q8_cache* c) { return size_t(c->n_blocks) * c->kv_heads * 4; }

// The shape of a cache (no pointers).
int q8_shape(const kvc_q8_cache* c, Q8* d) {
  if (c == nullptr) return KVC_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return KVC_EUNSUPPORTED;
  if (c->n_seqs < 0 || c->kv_heads < 1 || c->block_size < 1 || c->block_size > 4096 ||
      c->table_blocks < 1 || c->max_len < 0 || c->reserved != 0 || c->n_blocks < 1)
    return KVC_EINVAL;
  if (c->format != KVC_Q8_E4M3 && c->format != KVC_Q8_INT8) return KVC_EINVAL;
  if (int64_t(c->n_seqs) * c->kv_heads >= (int64_t(1) << 24)) return KVC_EINVAL;
  const int64_t room = int64_t(c->table_blocks) * c->block_size;
  if (room > (int64_t(1) << 30)) return KVC_EINVAL;
  if (c->n_blocks >= (int64_t(1) << 31) ||
      double(c->n_blocks) * c->kv_heads * c->block_size >= 4294967295.0)
    return KVC_EINVAL;
  d->B = c->n_seqs;
  d->H = c->kv_heads;
  d->D = c->head_dim;
  d->bs = c->block_size;
  d->tb = c->table_blocks;
  d->cap = c->max_len > 0 && c->max_len < room ? c->max_len : int(room);
  d->fmt = c->format;
  d->n_blocks = uint32_t(c->n_blocks);
  d->div = fast_div(uint32_t(c->block_size));
  d->k = static_cast<uint8_t*>(c->k_pool);
  d->v = static_cast<uint8_t*>(c->v_pool);
  d->ks = c->k_scale;
  d->vs = c->v_scale;
  d->table = c->table;
  d->seq_len = c->seq_len;
  return KVC_OK;
}

// Its pointers.
int q8_pointers(const kvc_q8_cache* c) {
  if (!c->k_pool || !c->v_pool || !c->k_scale || !c->v_scale || !c->table || !c->seq_len)
    return KVC_EINVAL;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(c->table, 4) || !aligned(c->seq_len, 4))
    return KVC_EALIGN;
  return KVC_OK;
}

// The cache's arrays as ranges: 0..3 pools and scales, 4..5 table and lengths.
void q8_ranges(const kvc_q8_cache* c, Range* r) {
  r[0] = {c->k_pool, pool_bytes(c)};
  r[1] = {c->v_pool, pool_bytes(c)};
  r[2] = {c->k_scale, scale_bytes(c)};
  r[3] = {c->v_scale, scale_bytes(c)};
  r[4] = {c->table, size_t(c->n_seqs) * c->table_blocks * 4};
  r[5] = {c->seq_len, size_t(c->n_seqs) * 4};
}

// Units of a launch that are counted in 32 bits.
bool too_many(uint64_t units) { return units > 0xffffff00ull; }

size_t attend_ws(const Q8& d, int rows) {
  const int pieces = q8_max_pieces(d.cap, rows);
  if (pieces == 1) return 0;
  const size_t n = size_t(d.B) * d.H * rows * pieces;
  return (n * (d.D + 2) * 4 + 255) & ~size_t(255);
}

int attend_shape(const kvc_q8_cache* c, int32_t group, int32_t window, Q8* d) {
  const int rc = q8_shape(c, d);
  if (rc != KVC_OK) return rc;
  if (group < 1 || window < 1) return KVC_EINVAL;
  if (group > 64) return KVC_EUNSUPPORTED;
  if (int64_t(group) * window > kMaxRows) return KVC_EINVAL;
  return KVC_OK;
}

int pages_shape(const kvc_page_table* t, Pages* p) {
  if (t == nullptr) return KVC_EINVAL;
  if (t->n_seqs < 0 || t->n_seqs > (1 << 20) || t->table_blocks < 1 || t->block_size < 1 ||
      t->block_size > 4096 || t->n_blocks < 1 || t->n_blocks > (1 << 24))
    return KVC_EINVAL;
  if (int64_t(t->table_blocks) * t->block_size > (int64_t(1) << 30)) return KVC_EINVAL;
  *p = Pages{t->n_seqs, t->table_blocks, t->block_size, t->n_blocks, t->table, t->seq_len, t->refs};
  return KVC_OK;
}

int pages_pointers(const kvc_page_table* t) {
  if (!t->table || !t->seq_len || !t->refs) return KVC_EINVAL;
  if (!aligned(t->table, 4) || !aligned(t->seq_len, 4) || !aligned(t->refs, 4)) return KVC_EALIGN;
  return KVC_OK;
}

void pages_ranges(const kvc_page_table* t, Range* r) {
  r[0] = {t->table, size_t(t->n_seqs) * t->table_blocks * 4};
  r[1] = {t->seq_len, size_t(t->n_seqs) * 4};
  r[2] = {t->refs, size_t(t->n_blocks) * 4};
}

constexpr int kMaxBufs = 4096;

int check_buffers(const kvc_page_buffer* bufs, int32_t n_bufs) {
  if (n_bufs < 0 || n_bufs > kMaxBufs || (n_bufs > 0 && !bufs)) return KVC_EINVAL;
  for (int i = 0; i < n_bufs; ++i)
    if (!bufs[i].base || bufs[i].page_bytes < 1 || bufs[i].page_bytes > (int64_t(1) << 32))
      return KVC_EINVAL;
  return KVC_OK;
}

// KVC_EINVAL if a buffer overlaps any of the n_r ranges or another buffer.  Sorted by
// address, only neighbours can overlap, and of a range only the buffers around it
// (all pairs took 10 us a call for 128 buffers and 9 ms for 4096; so 2 to 3 us and 0.2 ms).
int check_apart(const kvc_page_buffer* bufs, int n_bufs, int64_t n_blocks, const Range* r,
                int n_r) {
  struct Span {
    uintptr_t from, to;
  };
  constexpr int kFew = 64;
  Span few[kFew];
  Span* const s = n_bufs <= kFew ? few : new (std::nothrow) Span[n_bufs];
  if (!s) return KVC_EDEVICE;
  for (int i = 0; i < n_bufs; ++i) {
    const uintptr_t at = uintptr_t(bufs[i].base);
    s[i] = {at, at + size_t(bufs[i].page_bytes) * size_t(n_blocks)};
  }
  const auto before = [](const Span& a, const Span& b) { return a.from < b.from; };
  if (!std::is_sorted(s, s + n_bufs, before)) std::sort(s, s + n_bufs, before);
  bool alias = false;
  for (int i = 1; i < n_bufs; ++i) alias |= s[i - 1].to > s[i].from;
  for (int j = 0; j < n_r && !alias; ++j) {
    if (!r[j].p || r[j].n == 0) continue;
    const uintptr_t from = uintptr_t(r[j].p), to = from + r[j].n;
    // the last buffer that starts before the range ends
    const Span* z = std::lower_bound(s, s + n_bufs, Span{to, to}, before);
    alias = z != s && z[-1].to > from;
  }
  if (s != few) delete[] s;
  return alias ? KVC_EINVAL : KVC_OK;
}

// Groups of at most kMaxBuffers buffers with their chunks numbered through;
// one empty group when there are none.
int group_buffers(const kvc_page_buffer* bufs, int n_bufs, Buffers* groups) {
  int n = 0;
  for (int i0 = 0; i0 < n_bufs || n == 0; i0 += kMaxBuffers) {
    Buffers& g = groups[n++];
    g.n = n_bufs - i0 < kMaxBuffers ? n_bufs - i0 : kMaxBuffers;
    g.chunks = 0;
    for (int i = 0; i < g.n; ++i) {
      const kvc_page_buffer& b = bufs[i0 + i];
      const uint64_t bits = uint64_t(uintptr_t(b.base)) | uint64_t(b.page_bytes) | 16;
      g.b[i].base = static_cast<char*>(b.base);
      g.b[i].bytes = b.page_bytes;
      g.b[i].first = g.chunks;
      g.b[i].unit = uint32_t(bits & (~bits + 1));
      g.chunks += uint32_t((b.page_bytes + kCopyChunk - 1) / kCopyChunk);
    }
  }
  return n;
}

// A call's buffer groups, on the host.
struct Groups {
  Buffers* g;
  int n = 0;
  Groups(const kvc_page_buffer* bufs, int n_bufs)
      : g(new (std::nothrow) Buffers[n_bufs > 0 ? (n_bufs + kMaxBuffers - 1) / kMaxBuffers : 1]) {
    if (g) n = group_buffers(bufs, n_bufs, g);
  }
  ~Groups() { delete[] g; }
  Groups(const Groups&) = delete;
  Groups& operator=(const Groups&) = delete;
};

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

int kvc_q8_store(const kvc_q8_cache* c, int32_t T, int32_t t_stride, const int32_t* kept,
                 int32_t n_kept, const void* k, const void* v, void* stream) {
  Q8 d;
  int rc = q8_shape(c, &d);
  if (rc != KVC_OK) return rc;
  if (T < 1 || T > (1 << 27) || t_stride < T || (kept ? n_kept < 1 : n_kept != 0))
    return KVC_EINVAL;
  if (d.B == 0) return KVC_OK;
  if ((rc = q8_pointers(c)) != KVC_OK) return rc;
  if (!k || !v) return KVC_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || (kept && !aligned(kept, 4))) return KVC_EALIGN;
  const size_t nh = size_t(d.B) * d.H, rows = nh * size_t(t_stride) * d.D * 2;
  const int top = kept ? n_kept : T, slots = top < d.cap ? top : d.cap;
  if (too_many(nh * uint64_t((slots + d.bs - 1) / d.bs) * 2)) return KVC_EINVAL;
  Range r[6];
  q8_ranges(c, r);
  const Range in[] = {r[4], r[5], {k, rows}, {v, rows}, {kept, nh * size_t(n_kept) * 4}};
  if (any_alias(in, 5, r, 4)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_q8_store(d, T, t_stride, kept, n_kept, k, v, s);
  });
}

int kvc_q8_load(const kvc_q8_cache* c, int32_t T, int32_t t_stride, void* k_out, void* v_out,
                void* stream) {
  Q8 d;
  int rc = q8_shape(c, &d);
  if (rc != KVC_OK) return rc;
  if (T < 1 || T > (1 << 27) || t_stride < T) return KVC_EINVAL;
  if (d.B == 0) return KVC_OK;
  if ((rc = q8_pointers(c)) != KVC_OK) return rc;
  if (!k_out && !v_out) return KVC_EINVAL;
  if ((k_out && !aligned(k_out, 16)) || (v_out && !aligned(v_out, 16))) return KVC_EALIGN;
  const size_t rows = size_t(d.B) * d.H * size_t(t_stride) * d.D * 2;
  Range r[6];
  q8_ranges(c, r);
  const Range out[] = {{k_out, rows}, {v_out, rows}};
  if (any_alias(r, 6, out, 2)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_q8_load(d, T, t_stride, k_out, v_out, s);
  });
}

int kvc_q8_append(const kvc_q8_cache* c, int32_t window, const int32_t* n_new, const void* k_new,
                  const void* v_new, void* stream) {
  Q8 d;
  int rc = q8_shape(c, &d);
  if (rc != KVC_OK) return rc;
  if (window < 1 || window > (1 << 30)) return KVC_EINVAL;
  if (d.B == 0) return KVC_OK;
  if ((rc = q8_pointers(c)) != KVC_OK) return rc;
  if (!k_new || !v_new) return KVC_EINVAL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || (n_new && !aligned(n_new, 4)))
    return KVC_EALIGN;
  const size_t nh = size_t(d.B) * d.H, rows = nh * size_t(window) * d.D * 2;
  int64_t pages = (int64_t(window) + d.bs - 2) / d.bs + 1;
  if (pages > d.tb) pages = d.tb;
  if (too_many(nh * uint64_t(pages))) return KVC_EINVAL;
  Range r[6];
  q8_ranges(c, r);
  const Range in[] = {r[4], r[5], {k_new, rows}, {v_new, rows}, {n_new, size_t(d.B) * 4}};
  if (any_alias(in, 5, r, 4)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_q8_append(d, window, n_new, k_new, v_new, s);
  });
}

size_t kvc_q8_attend_workspace_bytes(const kvc_q8_cache* c, int32_t group, int32_t window) {
  Q8 d;
  if (attend_shape(c, group, window, &d) != KVC_OK) return size_t(-1);
  return attend_ws(d, group * window);
}

int kvc_q8_attend(const kvc_q8_cache* c, int32_t group, int32_t window, float scale,
                  const void* q, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  Q8 d;
  int rc = attend_shape(c, group, window, &d);
  if (rc != KVC_OK) return rc;
  if (!(scale >= 0.0f && scale <= 0x1p127f)) return KVC_EINVAL;  // scale * log2(e) is finite
  if (d.B == 0) return KVC_OK;
  if ((rc = q8_pointers(c)) != KVC_OK) return rc;
  if (!q || !out) return KVC_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4))) return KVC_EALIGN;
  const int R = group * window;
  const size_t need = attend_ws(d, R);
  if (need > 0 && (!ws || ws_bytes < need)) return KVC_EWORKSPACE;
  if (need > 0 && !aligned(ws, 256)) return KVC_EALIGN;
  const size_t rows = size_t(d.B) * d.H * R;
  Range r[7];
  q8_ranges(c, r);
  r[6] = {q, rows * d.D * 2};
  const Range out_r[] = {{out, rows * d.D * 2}, {lse, rows * 4}, {need > 0 ? ws : nullptr, need}};
  if (any_alias(r, 7, out_r, 3)) return KVC_EINVAL;
  const double f = scale != 0.0f ? double(scale) : 1.0 / sqrt(double(d.D));
  const float c_log2 = float(f * 1.4426950408889634);  // scale * log2(e)
  return launch_on(stream, [&](hipStream_t s) {
    return launch_q8_attend(d, group, window, c_log2, q, out, lse, static_cast<float*>(ws), s);
  });
}

size_t kvc_pages_workspace_bytes(const kvc_page_table* t, int32_t n_pairs) {
  Pages p;
  if (pages_shape(t, &p) != KVC_OK || n_pairs < 0 || n_pairs > (1 << 20)) return 0;
  return pages_ws(p, n_pairs).total * 4;
}

int kvc_pages_alloc(const kvc_page_table* t, const int32_t* want_len, int32_t* status, void* ws,
                    size_t ws_bytes, void* stream) {
  Pages p;
  int rc = pages_shape(t, &p);
  if (rc != KVC_OK) return rc;
  if (p.B == 0) return KVC_OK;
  if ((rc = pages_pointers(t)) != KVC_OK) return rc;
  if (!want_len || !status) return KVC_EINVAL;
  if (!aligned(want_len, 4) || !aligned(status, 4)) return KVC_EALIGN;
  if (!ws || ws_bytes < pages_ws(p, 0).total * 4) return KVC_EWORKSPACE;
  if (!aligned(ws, 256)) return KVC_EALIGN;
  const size_t per_seq = size_t(p.B) * 4;
  Range out[5];
  pages_ranges(t, out);
  out[3] = {status, per_seq};
  out[4] = {ws, ws_bytes};
  // the lengths are not touched, and are what a caller wants most often
  const Range in[] = {{want_len, per_seq}, out[1]};
  out[1] = Range{nullptr, 0};
  if (any_alias(in, 2, out, 5)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_pages_alloc(p, want_len, status, static_cast<int32_t*>(ws), s);
  });
}

int kvc_pages_fork(const kvc_page_table* t, int32_t n_pairs, const int32_t* src,
                   const int32_t* dst, const kvc_page_buffer* bufs, int32_t n_bufs,
                   int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  Pages p;
  int rc = pages_shape(t, &p);
  if (rc != KVC_OK) return rc;
  if (n_pairs < 0 || n_pairs > (1 << 20)) return KVC_EINVAL;
  if ((rc = check_buffers(bufs, n_bufs)) != KVC_OK) return rc;
  if (n_pairs == 0) return KVC_OK;
  if (p.B == 0) return KVC_EINVAL;
  if ((rc = pages_pointers(t)) != KVC_OK) return rc;
  if (!src || !dst || !status) return KVC_EINVAL;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4)) return KVC_EALIGN;
  if (!ws || ws_bytes < pages_ws(p, n_pairs).total * 4) return KVC_EWORKSPACE;
  if (!aligned(ws, 256)) return KVC_EALIGN;
  const size_t ids = size_t(n_pairs) * 4;
  Range out[7];
  pages_ranges(t, out);
  out[3] = {status, ids};
  out[4] = {ws, ws_bytes};
  const Range in[] = {{src, ids}, {dst, ids}};
  if (any_alias(in, 2, out, 5)) return KVC_EINVAL;
  out[5] = in[0];
  out[6] = in[1];
  if ((rc = check_apart(bufs, n_bufs, p.n, out, 7)) != KVC_OK) return rc;
  Groups g(bufs, n_bufs);
  if (!g.g) return KVC_EDEVICE;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_pages_fork(p, n_pairs, src, dst, g.g, g.n, status, static_cast<int32_t*>(ws), s);
  });
}

int kvc_pages_free(const kvc_page_table* t, int32_t n_ids, const int32_t* ids, void* stream) {
  Pages p;
  int rc = pages_shape(t, &p);
  if (rc != KVC_OK) return rc;
  if (n_ids < 0 || n_ids > (1 << 20)) return KVC_EINVAL;
  if (n_ids == 0 || p.B == 0) return KVC_OK;
  if ((rc = pages_pointers(t)) != KVC_OK) return rc;
  if (!ids) return KVC_EINVAL;
  if (!aligned(ids, 4)) return KVC_EALIGN;
  Range out[3];
  pages_ranges(t, out);
  const Range in[] = {{ids, size_t(n_ids) * 4}};
  if (any_alias(in, 1, out, 3)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) { return launch_pages_free(p, n_ids, ids, s); });
}

int kvc_pages_copy(int32_t n_blocks, int32_t n_pairs, const int32_t* src, const int32_t* dst,
                   const kvc_page_buffer* bufs, int32_t n_bufs, void* stream) {
  if (n_blocks < 1 || n_blocks > (1 << 24) || n_pairs < 0 || n_pairs > (1 << 24)) return KVC_EINVAL;
  int rc = check_buffers(bufs, n_bufs);
  if (rc != KVC_OK) return rc;
  if (n_pairs == 0 || n_bufs == 0) return KVC_OK;
  if (!src || !dst) return KVC_EINVAL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return KVC_EALIGN;
  const size_t ids = size_t(n_pairs) * 4;
  const Range in[] = {{src, ids}, {dst, ids}};
  if ((rc = check_apart(bufs, n_bufs, n_blocks, in, 2)) != KVC_OK) return rc;
  Groups g(bufs, n_bufs);
  if (!g.g) return KVC_EDEVICE;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_pages_copy(n_blocks, n_pairs, src, dst, g.g, g.n, s);
  });
}

int kvc_pages_compact(const kvc_page_table* t, const kvc_page_buffer* bufs, int32_t n_bufs,
                      int32_t* table_out, int32_t* refs_out, int32_t* remap, int32_t* n_live,
                      void* ws, size_t ws_bytes, void* stream) {
  Pages p;
  int rc = pages_shape(t, &p);
  if (rc != KVC_OK) return rc;
  if ((rc = check_buffers(bufs, n_bufs)) != KVC_OK) return rc;
  if (p.B == 0) return KVC_EINVAL;
  if ((rc = pages_pointers(t)) != KVC_OK) return rc;
  if (!table_out || !refs_out || !remap || !n_live) return KVC_EINVAL;
  if (!aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(remap, 4) || !aligned(n_live, 4))
    return KVC_EALIGN;
  if (!ws || ws_bytes < pages_ws(p, 0).total * 4) return KVC_EWORKSPACE;
  if (!aligned(ws, 256)) return KVC_EALIGN;
  Range all[8];
  pages_ranges(t, all);
  all[3] = {table_out, all[0].n};
  all[4] = {refs_out, all[2].n};
  all[5] = {remap, all[2].n};
  all[6] = {n_live, 4};
  all[7] = {ws, ws_bytes};
  if (any_alias(all, 3, all + 3, 5)) return KVC_EINVAL;
  if ((rc = check_apart(bufs, n_bufs, p.n, all, 8)) != KVC_OK) return rc;
  Groups g(bufs, n_bufs);
  if (!g.g) return KVC_EDEVICE;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_pages_compact(p, g.g, g.n, table_out, refs_out, remap, n_live,
                                static_cast<int32_t*>(ws), s);
  });
}

}  // extern "C"
