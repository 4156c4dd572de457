// Host side of the bf16 paged cache: validates every argument of its C entry points
// and enqueues the kernels.  No allocation on the device, no synchronisation, no
// global state.
#include <math.h>

#include "kvc_host.h"
#include "kvc_paged.h"

namespace kvc {
namespace {

constexpr int kMaxTokens = 1 << 23;   // a workgroup a token, the grid's limit
constexpr int64_t kMaxHeads = 1 << 24;   // query heads of a token: a workgroup counts their pieces in 31 bits
constexpr int64_t kMaxTokenStride = 1 << 24, kMaxHeadStride = int64_t(1) << 40;  // 64 tokens lie within 2^32 bytes

size_t pool_bytes(const kvc_paged_cache* c) {
  return size_t(c->n_blocks) * c->kv_heads * c->block_size * c->head_dim * 2;
}

// The shape of a cache (no pointers).
int paged_shape(const kvc_paged_cache* c, Paged* d) {
  if (c == nullptr) return KVC_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return KVC_EUNSUPPORTED;
  if (c->n_seqs < 0 || c->kv_heads < 1 || c->block_size < 1 || c->block_size > 4096 ||
      c->table_blocks < 1 || c->max_len < 0 || c->n_blocks < 1)
    return KVC_EINVAL;
  if (int64_t(c->n_seqs) * c->kv_heads >= (int64_t(1) << 24) || c->kv_heads >= (1 << 24))
    return KVC_EINVAL;
  const int64_t room = int64_t(c->table_blocks) * c->block_size;
  if (room > (int64_t(1) << 30)) return KVC_EINVAL;
  if (c->n_blocks >= (int64_t(1) << 31) ||
      double(c->n_blocks) * c->kv_heads * c->block_size >= 4294967295.0)
    return KVC_EINVAL;
  if (!c->weight != !c->pos) return KVC_EINVAL;
  d->B = c->n_seqs;
  d->H = c->kv_heads;
  d->D = c->head_dim;
  d->bs = c->block_size;
  d->tb = c->table_blocks;
  d->cap = c->max_len > 0 && c->max_len < room ? c->max_len : int(room);
  d->room = int(room);
  d->n_blocks = uint32_t(c->n_blocks);
  d->div = fast_div(uint32_t(c->block_size));
  d->k = static_cast<uint16_t*>(c->k_pool);
  d->v = static_cast<uint16_t*>(c->v_pool);
  d->table = c->table;
  d->seq_len = c->seq_len;
  d->weight = c->weight;
  d->pos = c->pos;
  return KVC_OK;
}

int paged_pointers(const kvc_paged_cache* c) {
  if (!c->k_pool || !c->v_pool || !c->table || !c->seq_len) return KVC_EINVAL;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->table, 4) ||
      !aligned(c->seq_len, 4) || !aligned(c->weight, 4) || !aligned(c->pos, 4))
    return KVC_EALIGN;
  return KVC_OK;
}

// The cache's arrays as ranges: 0..1 pools, 2..3 weight and pos, 4 table, 5 lengths.
void paged_ranges(const kvc_paged_cache* c, Range* r) {
  const size_t slots =
      size_t(c->n_seqs) * c->kv_heads * size_t(c->table_blocks) * size_t(c->block_size) * 4;
  r[0] = {c->k_pool, pool_bytes(c)};
  r[1] = {c->v_pool, pool_bytes(c)};
  r[2] = {c->weight, slots};
  r[3] = {c->pos, slots};
  r[4] = {c->table, size_t(c->n_seqs) * c->table_blocks * 4};
  r[5] = {c->seq_len, size_t(c->n_seqs) * 4};
}

// Rows of n tokens x heads, in bytes from p.
struct Span2 {
  const char* p;
  int64_t ts, hs;        // bytes
  int64_t n, heads, row;
  int64_t token() const { return (heads - 1) * hs + row; }  // extent of a token's rows
  int64_t all() const { return (n - 1) * ts + token(); }
};

int rows_ok(const kvc_rows* r, int64_t n, int64_t heads, int d, bool written, Rows* out, Span2* sp) {
  if (!r || !r->data) return KVC_EINVAL;
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > kMaxTokenStride ||
      r->head_stride > kMaxHeadStride)
    return KVC_EINVAL;
  if (!aligned(r->data, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return KVC_EALIGN;
  *out = {static_cast<uint16_t*>(r->data), r->token_stride, r->head_stride};
  *sp = {static_cast<const char*>(r->data), r->token_stride * 2, r->head_stride * 2, n, heads, int64_t(d) * 2};
  if (written) {
    const bool by_token = (heads == 1 || r->head_stride >= d) &&
                          (n == 1 || sp->ts >= sp->token());
    const bool by_head = (n == 1 || r->token_stride >= d) &&
                         (heads == 1 || sp->hs >= (n - 1) * sp->ts + sp->row);
    if (!by_token && !by_head) return KVC_EINVAL;
  }
  return KVC_OK;
}

// Whether two sets of rows share no byte as far as their strides tell: apart as ranges,
// or slices of the same tokens (one stride, each token's parts side by side).
bool rows_apart(const Span2& a, const Span2& b) {
  if (!overlap({a.p, size_t(a.all())}, {b.p, size_t(b.all())})) return true;
  if (a.ts != b.ts || a.ts <= 0 || a.token() > a.ts || b.token() > a.ts) return false;
  int64_t off = (b.p - a.p) % a.ts;
  if (off < 0) off += a.ts;
  return off >= a.token() && off + b.token() <= a.ts;
}
bool same_rows(const Span2& a, const Span2& b) {
  return a.p == b.p && (a.ts == b.ts || a.n == 1) && (a.hs == b.hs || a.heads == 1);
}
Range whole(const Span2& a) { return {a.p, size_t(a.all())}; }

int rope_ok(const kvc_rope_plan* f, int d, RopePlan* out) {
  if (!f || !f->freq) return KVC_EINVAL;
  if (f->rot_dim < 2 || f->rot_dim > d || f->rot_dim % 2 != 0 || f->reserved != 0 ||
      (f->interleaved != 0 && f->interleaved != 1) || !isfinite(f->mscale))
    return KVC_EINVAL;
  if (!aligned(f->freq, 8)) return KVC_EALIGN;
  *out = {f->freq, f->rot_dim, f->interleaved, f->mscale, 1.0f};
  return KVC_OK;
}

// What kvc_paged_attend and its workspace are asked for (no pointers).
int attend_shape(const kvc_paged_cache* c, int32_t group, int32_t n_tokens, int32_t max_new, Paged* d,
                 Chunks* k) {
  const int rc = paged_shape(c, d);
  if (rc != KVC_OK) return rc;
  if (group < 1 || n_tokens < 0 || n_tokens > kMaxTokens || max_new < 0) return KVC_EINVAL;
  if (group > 64) return KVC_EUNSUPPORTED;
  if (int64_t(group) * d->H > kMaxHeads || int64_t(n_tokens) * group * d->H >= (int64_t(1) << 30))
    return KVC_EINVAL;
  *k = {nullptr, d->B, n_tokens, max_new > 0 && max_new < n_tokens ? max_new : n_tokens};
  if (int64_t(group) * k->max_new > kFewRows &&   // workgroups of a launch
      (int64_t(first_slot(n_tokens, d->B, group, tile_max_pieces(d->cap))) * d->H >= (int64_t(1) << 23) ||
       int64_t(first_tile(n_tokens, d->B, group)) * d->H >= (int64_t(1) << 23)))
    return KVC_EINVAL;
  return KVC_OK;
}

// What kvc_paged_evict and its workspace are asked for (no pointers).  A launch has
// below 2^32 work-items, and a long head is planned by 1024 of them.
int evict_shape(const kvc_paged_cache* c, int32_t budget, Paged* d) {
  const int rc = paged_shape(c, d);
  if (rc != KVC_OK) return rc;
  return budget < 1 || int64_t(d->B) * d->H >= (int64_t(1) << 22) ? KVC_EINVAL : KVC_OK;
}

bool scale_ok(float scale) { return scale >= 0.0f && scale <= 0x1p127f; }
float in_log2(float scale, int d) {
  const double f = scale != 0.0f ? double(scale) : 1.0 / sqrt(double(d));
  return float(f * 1.4426950408889634);
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

int kvc_rope(int32_t n_tokens, int32_t heads, int32_t head_dim, const kvc_rope_plan* rope,
             int32_t backward, const int32_t* positions, const kvc_rows* x, const kvc_rows* y,
             void* stream) {
  if (head_dim != 64 && head_dim != 128) return KVC_EUNSUPPORTED;
  if (n_tokens < 0 || n_tokens > kMaxTokens || heads < 1 || heads > (1 << 16) ||
      int64_t(n_tokens) * heads >= (int64_t(1) << 30) || (backward != 0 && backward != 1))
    return KVC_EINVAL;
  RopePlan f;
  int rc = rope_ok(rope, head_dim, &f);
  if (rc != KVC_OK) return rc;
  if (n_tokens == 0) return KVC_OK;
  f.sign = backward ? -1.0f : 1.0f;
  Rows rx, ry;
  Span2 sx, sy;
  if ((rc = rows_ok(x, n_tokens, heads, head_dim, false, &rx, &sx)) != KVC_OK) return rc;
  if ((rc = rows_ok(y, n_tokens, heads, head_dim, true, &ry, &sy)) != KVC_OK) return rc;
  if (!positions) return KVC_EINVAL;
  if (!aligned(positions, 4)) return KVC_EALIGN;
  if (!same_rows(sx, sy) && !rows_apart(sx, sy)) return KVC_EINVAL;
  const Range out = whole(sy);
  if (overlap(out, {positions, size_t(n_tokens) * 4}) || overlap(out, {f.freq, size_t(f.r / 2) * 8}))
    return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_rope(f, n_tokens, heads, head_dim, positions, rx, ry, s);
  });
}

int kvc_paged_append(const kvc_paged_cache* c, int32_t n_tokens, const int32_t* starts,
                     const int32_t* positions, const kvc_rope_plan* rope, int32_t group,
                     const kvc_rows* q, const kvc_rows* q_out, const kvc_rows* k,
                     const kvc_rows* v, void* stream) {
  Paged d;
  int rc = paged_shape(c, &d);
  if (rc != KVC_OK) return rc;
  if (n_tokens < 0 || n_tokens > kMaxTokens || int64_t(n_tokens) * d.H >= (int64_t(1) << 30))
    return KVC_EINVAL;
  RopePlan f{nullptr, 0, 0, 1.0f, 1.0f};
  if (rope && (rc = rope_ok(rope, d.D, &f)) != KVC_OK) return rc;
  if (q && (!rope || group < 1)) return KVC_EINVAL;
  if (q && group > 64) return KVC_EUNSUPPORTED;
  if (!q && q_out) return KVC_EINVAL;
  if (q && (int64_t(group) * d.H > kMaxHeads || int64_t(n_tokens) * group * d.H >= (int64_t(1) << 30)))
    return KVC_EINVAL;
  if (d.B == 0 || n_tokens == 0) return KVC_OK;
  if ((rc = paged_pointers(c)) != KVC_OK) return rc;
  if (!starts) return KVC_EINVAL;
  if (!aligned(starts, 4) || !aligned(positions, 4)) return KVC_EALIGN;
  Rows rq{}, ro{}, rk, rv;
  Span2 sq{}, so{}, sk, sv;
  if ((rc = rows_ok(k, n_tokens, d.H, d.D, false, &rk, &sk)) != KVC_OK) return rc;
  if ((rc = rows_ok(v, n_tokens, d.H, d.D, false, &rv, &sv)) != KVC_OK) return rc;
  const int q_heads = q ? group * d.H : 0;
  if (q) {
    if ((rc = rows_ok(q, n_tokens, q_heads, d.D, false, &rq, &sq)) != KVC_OK) return rc;
    if ((rc = rows_ok(q_out, n_tokens, q_heads, d.D, true, &ro, &so)) != KVC_OK) return rc;
  }
  Range r[6];
  paged_ranges(c, r);
  const Range in[] = {r[4], r[5], {starts, size_t(d.B + 1) * 4}, {positions, size_t(n_tokens) * 4},
                      {f.freq, size_t(f.r / 2) * 8}, whole(sk), whole(sv), q ? whole(sq) : Range{nullptr, 0}};
  if (any_alias(in, 8, r, 4)) return KVC_EINVAL;   // the cache against all inputs
  if (q) {
    const Range out = whole(so);
    for (int i = 0; i < 5; ++i)
      if (overlap(out, in[i])) return KVC_EINVAL;
    for (int i = 0; i < 4; ++i)
      if (overlap(out, r[i])) return KVC_EINVAL;
    if (!rows_apart(so, sk) || !rows_apart(so, sv)) return KVC_EINVAL;
    if (!same_rows(so, sq) && !rows_apart(so, sq)) return KVC_EINVAL;
  }
  const Chunks ch{starts, d.B, n_tokens, n_tokens};
  return launch_on(stream, [&](hipStream_t s) {
    return launch_paged_append(d, ch, positions, f, q_heads, rq, ro, rk, rv, s);
  });
}

size_t kvc_paged_attend_workspace_bytes(const kvc_paged_cache* c, int32_t group, int32_t n_tokens,
                                        int32_t max_new) {
  Paged d;
  Chunks k;
  if (attend_shape(c, group, n_tokens, max_new, &d, &k) != KVC_OK) return size_t(-1);
  return attend_ws(d, k, group).total * 4;
}

int kvc_paged_attend(const kvc_paged_cache* c, int32_t group, int32_t n_tokens, int32_t max_new,
                     const int32_t* starts, float scale, const kvc_rows* q, const kvc_rows* out,
                     float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttendCall a{};
  int rc = attend_shape(c, group, n_tokens, max_new, &a.c, &a.k);
  if (rc != KVC_OK) return rc;
  if (!scale_ok(scale)) return KVC_EINVAL;
  const Paged& d = a.c;
  if (d.B == 0 || n_tokens == 0) return KVC_OK;
  if ((rc = paged_pointers(c)) != KVC_OK) return rc;
  if (!starts) return KVC_EINVAL;
  if (!aligned(starts, 4) || !aligned(lse, 4)) return KVC_EALIGN;
  Span2 sq, so;
  const int heads = group * d.H;
  if ((rc = rows_ok(q, n_tokens, heads, d.D, false, &a.q, &sq)) != KVC_OK) return rc;
  if ((rc = rows_ok(out, n_tokens, heads, d.D, true, &a.out, &so)) != KVC_OK) return rc;
  const size_t need = attend_ws(d, a.k, group).total * 4;
  if (need > 0 && (!ws || ws_bytes < need)) return KVC_EWORKSPACE;
  if (need > 0 && !aligned(ws, 256)) return KVC_EALIGN;
  Range r[8];
  paged_ranges(c, r);
  r[6] = {starts, size_t(d.B + 1) * 4};
  const Range outs[] = {whole(so), {lse, size_t(n_tokens) * heads * 4}, {need > 0 ? ws : nullptr, need}};
  if (any_alias(r, 7, outs, 3)) return KVC_EINVAL;
  // q may be a slice beside out, never under the others; weights grow, all else is read
  if (!rows_apart(so, sq) || overlap(whole(sq), outs[1]) || overlap(whole(sq), outs[2])) return KVC_EINVAL;
  const Range in[] = {r[0], r[1], r[3], r[4], r[5], r[6], whole(sq)};
  if (any_alias(in, 7, &r[2], 1)) return KVC_EINVAL;
  a.k.starts = starts;
  a.G = group;
  a.c_log2 = in_log2(scale, d.D);
  a.lse = lse;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_paged_attend(a, static_cast<float*>(ws), s);
  });
}

int kvc_prompt_attend(int32_t n_seqs, int32_t kv_heads, int32_t group, int32_t head_dim,
                      int32_t n_tokens, const int32_t* starts, float scale, const kvc_rows* q,
                      const kvc_rows* k, const kvc_rows* v, const kvc_rows* out, float* lse,
                      void* stream) {
  if (head_dim != 64 && head_dim != 128) return KVC_EUNSUPPORTED;
  if (n_seqs < 0 || kv_heads < 1 || kv_heads > (1 << 16) || group < 1 || n_tokens < 0 ||
      n_tokens > kMaxTokens || !scale_ok(scale))
    return KVC_EINVAL;
  if (group > 64) return KVC_EUNSUPPORTED;
  const int64_t heads = int64_t(group) * kv_heads;
  if (n_tokens * heads >= (int64_t(1) << 30) || int64_t(n_seqs) * kv_heads >= (int64_t(1) << 22))
    return KVC_EINVAL;
  if (n_seqs == 0 || n_tokens == 0) return KVC_OK;
  if (!starts) return KVC_EINVAL;
  if (!aligned(starts, 4) || !aligned(lse, 4)) return KVC_EALIGN;
  Rows rq, rk, rv, ro;
  Span2 sq, sk, sv, so;
  int rc;
  if ((rc = rows_ok(q, n_tokens, heads, head_dim, false, &rq, &sq)) != KVC_OK) return rc;
  if ((rc = rows_ok(k, n_tokens, kv_heads, head_dim, false, &rk, &sk)) != KVC_OK) return rc;
  if ((rc = rows_ok(v, n_tokens, kv_heads, head_dim, false, &rv, &sv)) != KVC_OK) return rc;
  if ((rc = rows_ok(out, n_tokens, heads, head_dim, true, &ro, &so)) != KVC_OK) return rc;
  const Range st{starts, size_t(n_seqs + 1) * 4}, ls{lse, size_t(n_tokens) * heads * 4};
  if (overlap(whole(so), st) || overlap(ls, st) || overlap(whole(so), ls) || !rows_apart(so, sq) ||
      !rows_apart(so, sk) || !rows_apart(so, sv) || overlap(ls, whole(sq)) || overlap(ls, whole(sk)) ||
      overlap(ls, whole(sv)))
    return KVC_EINVAL;
  const Chunks ch{starts, n_seqs, n_tokens, n_tokens};
  return launch_on(stream, [&](hipStream_t s) {
    return launch_prompt_attend(kv_heads, group, head_dim, ch, in_log2(scale, head_dim), rq, rk, rv, ro, lse, s);
  });
}

size_t kvc_paged_evict_workspace_bytes(const kvc_paged_cache* c, int32_t budget) {
  Paged d;
  if (evict_shape(c, budget, &d) != KVC_OK) return 0;
  const size_t n = evict_ws(d, budget);
  return n > 0 ? n : 256;
}

int kvc_paged_evict(const kvc_paged_cache* c, const int32_t* seen, int32_t budget, int32_t sinks,
                    int32_t recent, void* ws, size_t ws_bytes, void* stream) {
  Paged d;
  int rc = evict_shape(c, budget, &d);
  if (rc != KVC_OK) return rc;
  if (sinks < 0 || recent < 0) return KVC_EINVAL;
  if (d.B == 0) return KVC_OK;
  if ((rc = paged_pointers(c)) != KVC_OK) return rc;
  if (!c->weight || !seen) return KVC_EINVAL;
  if (!aligned(seen, 4)) return KVC_EALIGN;
  const size_t need = evict_ws(d, budget);
  if (!ws || ws_bytes < need) return KVC_EWORKSPACE;
  if (!aligned(ws, 256)) return KVC_EALIGN;
  Range r[7];
  paged_ranges(c, r);
  const Range in[] = {r[4], {seen, size_t(d.B) * 4}};
  const Range out[] = {r[0], r[1], r[2], r[3], r[5], {ws, need}};
  if (any_alias(in, 2, out, 6)) return KVC_EINVAL;
  return launch_on(stream, [&](hipStream_t s) {
    return launch_paged_evict(d, seen, budget, sinks, recent, static_cast<int32_t*>(ws), s);
  });
}

}  // extern "C"
