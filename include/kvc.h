/*
 * kvc.h -- C ABI of libkvc: the decode-time KV-cache compression event
 * (adaptive mass-segmented selection) on AMD MI355X (gfx950).
 *
 * Sources.  The operation is the event described in the notes on
 * "Adaptive Mass-Segmented KV Compression for Long-Form Reasoning" (AMS):
 * section 整体框架 (overall framework) says selection runs independently for
 * every layer and KV head on the current cache and yields a compact cache of
 * the target budget; 关键设计 1-4 (key designs 1-4) give the mass, the
 * cumulative-mass cuts, the segment quotas and the in-segment selection with
 * gather-and-compact.  The one-segment special case is the max-pooled global
 * top-K of the notes on "RefreshKV: Updating Small KV Cache During Long-form
 * Generation" (A2 method details, prefill stage; A6 appendix, baselines).
 *
 * Conventions shared by every entry point.
 *  - One call covers n_heads independent head-events (layer x batch x KV
 *    head).  Head n's data is the n-th slab of every array.
 *  - Every pointer except `params` and the returned strings is a DEVICE
 *    pointer owned by the caller.  The library allocates no memory, keeps no
 *    state between calls and never synchronises: all work is enqueued on
 *    `stream` (a hipStream_t passed as void*; NULL = the null stream) and
 *    completes asynchronously.  Results are deterministic: the same inputs
 *    give the same bits on every run, and a head's results do not depend on
 *    the other heads of the call (a head alone, with T set to its real
 *    length, gives the bits it gets inside a left-padded batch).
 *  - All arguments are validated on the host before anything is enqueued; on
 *    an error return nothing has been launched and no output was touched.
 *  - A call enqueues kernel launches only (no memset, copy or allocation), so
 *    it can be captured into a HIP graph and replayed with new inputs copied
 *    into the captured buffers.
 *  - Return values: KVC_OK (0), KVC_NOOP (1, informational: T <= budget, so
 *    nothing is evicted), negative = error (see kvc_strerror).
 *  - bf16 tensors are raw IEEE bfloat16; q, k, v, k_out, v_out must be
 *    16-byte aligned; fp32/u64/i32 arrays need their natural alignment.
 *  - Outputs may not overlap inputs (KVC_EINVAL).
 *  - Calls that share a workspace or outputs must be ordered on one stream.
 *  - Precondition (not checked): q and k are finite.
 *
 * Array layouts (row-major, innermost last; NH = n_heads, G = group,
 * W = window, d = head_dim, S = kvc_segment_capacity(p)):
 *   q_win      bf16 [NH][G][W][d]     last W queries of the G query heads
 *                                      that share each KV head (post-RoPE);
 *                                      window query w sits at position T-W+w
 *   k, v       bf16 [NH][t_stride][d] cached keys/values, rows >= T unused
 *   u          f32  [NH][T]            window usage (step 1 output)
 *   score      f32  [NH][T]            pooled usage, the base score
 *   credit_in  u64  [NH][n_prev]       carried EMA credit, Q44 fixed point
 *   credit_upd u64  [NH][T]            updated credit per position, Q44
 *   seg_start  i32  [NH][S]            first position of each segment
 *   seg_quota  i32  [NH][S]            positions to pick in each segment
 *   n_seg      i32  [NH]               segments used per head
 *   kept       i32  [NH][budget]       kept positions, ascending; -1 pads the
 *                                      tail only when T < budget
 *   k_out,v_out bf16 [NH][budget][d]   compacted cache (zero rows past T)
 *   credit_out u64  [NH][budget]       credit of the kept positions
 */
#ifndef KVC_H
#define KVC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVC_ABI_VERSION 3

enum kvc_status {
  KVC_OK = 0,
  KVC_NOOP = 1,           /* T <= budget: kept = 0..T-1, identity copy      */
  KVC_EINVAL = -1,        /* a shape or parameter is out of range, a
                             required pointer is NULL, or outputs alias
                             inputs                                          */
  KVC_EALIGN = -2,        /* a pointer is not aligned as required           */
  KVC_EWORKSPACE = -3,    /* ws is NULL or ws_bytes < kvc_workspace_bytes() */
  KVC_EUNSUPPORTED = -4,  /* head_dim or group outside the built variants   */
  KVC_EDEVICE = -5,       /* the HIP runtime reported a launch error        */
  KVC_ESCRATCH = -6       /* kvc_compress_event_noalloc: the event needs more
                             scratch than KVC_NOALLOC_SCRATCH_BYTES          */
};

/* 8-bit formats of a paged cache. */
enum { KVC_Q8_E4M3 = 0, KVC_Q8_INT8 = 1 };

/* Scratch held on each GPU by kvc_compress_event_noalloc (64 MiB). */
#define KVC_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

enum { KVC_POOL_AVG = 0, KVC_POOL_MAX = 1 };
enum { KVC_AGG_SUM = 0, KVC_AGG_MAX = 1 };
enum { KVC_QUOTA_MASS = 0, KVC_QUOTA_UNIFORM = 1 };

/* Event parameters, named after the pages' quantities.  Field order fixes the
 * layout: 17 int32, one float, four doubles, two int32, then one pointer
 * (120 bytes, no padding). */
typedef struct kvc_params {
  int32_t n_heads;     /* NH independent head-events; 0 = nothing to do      */
  int32_t group;       /* G query heads per KV head, 1..64                   */
  int32_t head_dim;    /* d, 64 or 128                                       */
  int32_t T;           /* valid cached positions per head, 1..2^18           */
  int32_t t_stride;    /* rows allocated per head in k/v (>= T)              */
  int32_t window;      /* W recent queries, 1..T; W*G <= 4096 and
                          G*ceil(W/32)*32 <= 4096 (32-row MFMA blocks per
                          query head); F*W*W*G < 2^22 with F = 2 for
                          average pooling and F = pool_kernel for max
                          pooling keeps the fixed-point usage totals below
                          2^63 (step 1's usage sums to at most W*W*G per
                          head, and pooling multiplies that by < F)        */
  int32_t budget;      /* K positions kept per head, >= 1                    */
  int32_t seg_min;     /* shortest segment after merging (>= 1), e.g. 16     */
  int32_t seg_max;     /* longest segment after splitting, e.g. 256; 0 = none*/
  int32_t q_min;       /* per-segment minimum quota (>= 0), e.g. 1           */
  int32_t sinks;       /* leading must-keep positions (>= 0), e.g. 4         */
  int32_t recent;      /* trailing must-keep positions (>= 0), e.g. 64       */
  int32_t pool_kernel; /* odd pooling width 1..63, e.g. 7                    */
  int32_t pool_mode;   /* KVC_POOL_AVG (AMS) or KVC_POOL_MAX (SnapKV-style)  */
  int32_t head_agg;    /* KVC_AGG_SUM or KVC_AGG_MAX over the G query heads  */
  int32_t ema;         /* 1 = EMA credit on, 0 = off                         */
  int32_t n_prev;      /* credit entries carried per head (0..T; 0 if !ema)  */
  float scale;         /* softmax scale; 0 => 1/sqrt(head_dim); otherwise
                          finite with scale*log2(e) >= 2^-60                 */
  double delta;        /* target segment mass Delta in (0, inf); >= 1 => no
                          mass cuts; at most 1024 thresholds                 */
  double lambda;       /* EMA decay, [0,1], e.g. 0.9                          */
  double beta;         /* weight of the current mass, [0,1], e.g. 0.9        */
  double eps;          /* mass floor epsilon, (0, 1], e.g. 1e-6              */
  int32_t seg_fixed;   /* 0 = cuts from the cumulative mass (the method);
                          L > 0 = ablation "fixed-length segments" [AMS
                          notes, ablations, Table 7]: raw segments of L
                          positions (the last one shorter), then merge and
                          split as usual; ceil(T/L) <= 1025              */
  int32_t quota_mode;  /* KVC_QUOTA_MASS (the method) or KVC_QUOTA_UNIFORM:
                          ablation "no mass-weighted quota" [same table]:
                          every segment weighs 1 in the share of the
                          remainder and in the redistribution order      */
  const int32_t* valid_len; /* NULL, or a DEVICE array [n_heads] for ragged
                          (left-padded) batches [SkipKV notes, observation 1
                          and §4.1, attention mask M]: head n holds padding
                          at positions [0, T-len) and real tokens at
                          [T-len, T), len = valid_len[n] clamped to [W, T].
                          The event runs on the real tokens only, exactly
                          as on a cache of length len: u, score and
                          credit_upd are 0 on the padding, seg_start and
                          kept are positions of the padded cache, kept
                          holds min(budget, len) positions, and
                          credit_in[n][j] is the credit of position
                          T-len+j (j < min(n_prev, len)).  With valid_len
                          set, KVC_NOOP is never returned: a head with
                          len <= budget gets its identity copy and the
                          call returns KVC_OK.                            */
} kvc_params;

/* Step 1: window score [AMS notes, key design 1: usage of the most recent W
 * queries per cached position, partly observed suffix filled with the window
 * maximum; SkipKV notes §4.1: softmax(QK^T/sqrt(d)) over an observation window
 * with GQA head mapping].
 * u[n][t] = AGG_g sum_{w : T-W+w >= t} softmax_t'(scale*<q[n][g][w], k[n][t']>)
 * over t' <= T-W+w (AGG = sum or max over g of the per-head sums), then
 * u[n][t] = max_{t' <= T-W} u[n][t'] for t > T-W.  fp32 output; bf16 matrix
 * products with fp32 accumulation, fp32 softmax.
 * ws: at least kvc_workspace_bytes(p). */
int kvc_score_window(const kvc_params* p, const void* q_win, const void* k, float* u,
                     void* ws, size_t ws_bytes, void* stream);

/* Step 2 + step 3: mass, prefix and segmentation with quotas [AMS notes, key
 * design 1 (mass eq. m_i = (max(u_i,0)+eps)/sum, EMA eq.), key design 2 (C(t),
 * b_k = min{t : C(t) >= k*Delta}, split/merge to seg_min/seg_max), key
 * design 3 (must-keep sinks + recent suffix, q_i^min = min(q_min, L_i),
 * remainder split by segment mass with rounding, clip and redistribute)].
 * score[n][t] = pooled u (avg or max over pool_kernel in-range neighbours).
 * With ema: credit_in (may be NULL only when n_prev == 0) is the carried
 * credit of positions 0..n_prev-1; credit_upd receives the updated credit of
 * every position (required when ema, ignored otherwise).
 * Outputs seg_start/seg_quota/n_seg as laid out above.  Integer decisions
 * follow an exact fixed-point contract, bit-identical to a sequential
 * evaluation.  Returns KVC_NOOP (n_seg = 0) when T <= budget.
 * Precondition on u (not checked: it lives on the device): finite,
 * non-negative values whose pooled sum per head is at most F*W*W*G (the bound
 * on `window` above) -- which every u written by kvc_score_window satisfies.
 * Out-of-range values are clamped to [0, 2^23] (NaN to 0) before the
 * fixed-point conversion, so any input gives a valid partition, quotas that
 * respect the segment lengths and in-range indices; but a pooled sum past
 * 2^23 wraps the 64-bit fixed-point totals and the cuts and quotas are then
 * not the method's. */
int kvc_mass_segment(const kvc_params* p, const float* u, const uint64_t* credit_in,
                     float* score, uint64_t* credit_upd, int32_t* seg_start,
                     int32_t* seg_quota, int32_t* n_seg, void* ws, size_t ws_bytes,
                     void* stream);

/* Step 4: select [AMS notes, key design 3, last paragraph: union with the
 * must-keep set counting duplicates once, over budget drop low-score picks,
 * under budget add high-score unselected positions; key design 4: per-segment
 * top-k on a base score of shape [B,Hkv,T], kept indices sorted].
 * score: any finite fp32 base score (the pooled usage by default).  In each
 * segment the min(quota, candidates) non-must-keep positions with the largest
 * score are picked, ties to the lower position; the result always holds
 * min(budget, T) positions in ascending order.  Returns KVC_NOOP (kept =
 * 0..T-1, -1 padded) when T <= budget. */
int kvc_select(const kvc_params* p, const float* score, const int32_t* seg_start,
               const int32_t* seg_quota, const int32_t* n_seg, int32_t* kept, void* ws,
               size_t ws_bytes, void* stream);

/* Step 5: gather-and-compact [AMS notes, key design 4: the same kept indices
 * gather K and V into a fixed-length per-head cache; key design 1, last
 * paragraph: the credit follows the kept positions].
 * k_out[n][j] = k[n][kept[n][j]], v_out likewise, credit_out[n][j] =
 * credit_upd[n][kept[n][j]] (both credit pointers NULL, or both set); rows
 * with kept = -1 are zero-filled.  Bitwise copies; no workspace. */
int kvc_gather_compact(const kvc_params* p, const int32_t* kept, const void* k, const void* v,
                       const uint64_t* credit_upd, void* k_out, void* v_out,
                       uint64_t* credit_out, void* stream);

/* Step 5 on a paged cache [AMS notes, key design 4, appendix E paragraph:
 * the runtime allocates new blocks, copies each head's KV from its kept
 * original positions into the new physical slots, swaps the request's block
 * table and frees the old blocks; one compacted slot may hold KV from
 * different original positions in different heads].
 * Pools: k_pool, v_pool (source) and k_pool_out, v_pool_out (destination,
 * may be the same allocations) are bf16 [n_blocks][kv_heads][block_size][d].
 * Head n = b * kv_heads + h (n_heads = B * kv_heads); logical position t of
 * sequence b lives in block table_in[b][t / block_size], slot t % block_size
 * (table_in is i32 [B][table_in_blocks], table_in_blocks >= ceil(T /
 * block_size)).  Slot j of the compacted cache goes to block
 * table_out[b][j / block_size], slot j % block_size (i32 [B][table_out_blocks],
 * table_out_blocks >= ceil(budget / block_size)): for head h it receives the
 * row of position kept[n][j], or zeros where kept is -1.  Blocks named in
 * table_out must not appear in table_in (the copy reads old blocks while
 * writing new ones); no other block is written.  Block ids outside
 * [0, n_blocks) are never dereferenced (the destination row is skipped, a bad
 * source reads as zeros).  credit_upd/credit_out are optional and as in
 * kvc_gather_compact.  Swapping the tables and freeing the old blocks are the
 * caller's; nothing here allocates. */
int kvc_gather_paged(const kvc_params* p, int32_t kv_heads, int32_t block_size, int64_t n_blocks,
                     const int32_t* kept, const void* k_pool, const void* v_pool,
                     const int32_t* table_in, int32_t table_in_blocks, const int32_t* table_out,
                     int32_t table_out_blocks, void* k_pool_out, void* v_pool_out,
                     const uint64_t* credit_upd, uint64_t* credit_out, void* stream);

/* RefreshKV decode-loop pieces [notes on "RefreshKV: Updating Small KV Cache
 * During Long-form Generation", A2 method details: a full cache C_f and a
 * partial cache C_p of K entries per head; every S steps a query comparison
 * per layer (cosine of the current query averaged over the layer's query
 * heads against the one of its last full-attention step, full step when
 * below the threshold s); partial steps append the new token to C_p and drop
 * the entry with the lowest score of the last full step; a full step first
 * writes the tokens decoded with C_p into C_f, then refreshes C_p (the
 * one-segment event on C_f followed by kvc_partial_init)].  The caller runs
 * the loop and decides when to call what. */

/* Query comparison for `rows` (layer, sequence) rows.  q: bf16
 * [rows][heads_q][head_dim], the current token's queries (head_dim 64 or
 * 128).  q_ref: f64 [rows][head_dim], the head sums of each row's last full
 * step (the cosine is scale-invariant, so sums decide as means do); read,
 * and where a row fires and update_ref != 0, overwritten with the current
 * head sum.  full: i32 [rows], 1 where cos < threshold (a zero vector counts
 * as cos = 1).  cos_out: optional f64 [rows].  fp64 arithmetic. */
int kvc_qc_trigger(int32_t rows, int32_t heads_q, int32_t head_dim, const void* q, double* q_ref,
                   double threshold, int32_t update_ref, int32_t* full, double* cos_out,
                   void* stream);

/* C_p bookkeeping after a refresh: part_pos[n][j] = kept[n][j] and
 * part_score[n][j] = score[n][kept[n][j]] (+inf where kept is -1), with
 * kept/score as produced by the event (f32 score [NH][T], i32 kept
 * [NH][budget]); part_score f32 and part_pos i32 are [NH][budget]. */
int kvc_partial_init(const kvc_params* p, const int32_t* kept, const float* score,
                     float* part_score, int32_t* part_pos, void* stream);

/* One partial step for every head: the slot with the lowest part_score
 * (first slot on ties; scores must not be NaN) receives k_new[n], v_new[n]
 * (bf16 [n_heads][head_dim]) in k_part, v_part (bf16 [n_heads][K][head_dim]);
 * its score becomes +inf and its position t_new.  evicted: i32 [n_heads],
 * the slot used. */
int kvc_partial_append(int32_t n_heads, int32_t K, int32_t head_dim, float* part_score,
                       int32_t* part_pos, void* k_part, void* v_part, const void* k_new,
                       const void* v_new, int32_t t_new, int32_t* evicted, void* stream);

/* Full step, first half: every C_p slot with t_from <= part_pos < t_stride
 * is copied to row part_pos of k_full, v_full (bf16 [n_heads][t_stride]
 * [head_dim]); other rows are untouched. */
int kvc_full_sync(int32_t n_heads, int32_t K, int32_t head_dim, const int32_t* part_pos,
                  const void* k_part, const void* v_part, int32_t t_from, int32_t t_stride,
                  void* k_full, void* v_full, void* stream);

/* The whole event, steps 1-5 in one enqueue [AMS notes, overall framework].
 * credit_in/credit_out as above (credit_out required when ema); u_out (may be
 * NULL) receives the step-1 usage.  kept_out receives the kept positions.
 * Equals kvc_score_window -> kvc_mass_segment -> kvc_select ->
 * kvc_gather_compact on the same arguments, bit for bit.
 * The caller keeps counting logical (RoPE) positions from its generation
 * count; the compacted cache changes only the physical slots [AMS notes,
 * key design 4, appendix E paragraph]. */
int kvc_compress_event(const kvc_params* p, const void* q_win, const void* k, const void* v,
                       const uint64_t* credit_in, void* k_out, void* v_out,
                       uint64_t* credit_out, int32_t* kept_out, float* u_out, void* ws,
                       size_t ws_bytes, void* stream);

/* The whole event exactly as kvc_compress_event (same arguments, same
 * results, bit for bit), for callers that cannot allocate device memory:
 * code under HIP graph capture, serving loops and harnesses that forbid
 * allocation.  Instead of a workspace argument it uses scratch memory the
 * library holds on each GPU from module load until the process ends: a
 * device array of KVC_NOALLOC_SCRATCH_BYTES.  Events whose
 * kvc_workspace_bytes() exceeds that return KVC_ESCRATCH before anything is
 * enqueued (the Qwen-7B-shaped 1792-head event needs about 29 MB; larger
 * events use kvc_compress_event with a workspace).  Nothing is allocated and
 * nothing is freed.  The GPU is the one `stream` runs on (the current device
 * for the NULL stream); the first call on a GPU looks the array's address up
 * once.  Every call on one GPU shares that GPU's array and leaves its
 * contents behind (no call relies on them): calls that overlap in time on
 * one GPU -- different streams, or different host threads without ordering
 * -- race on it and must not be issued. */
int kvc_compress_event_noalloc(const kvc_params* p, const void* q_win, const void* k,
                               const void* v, const uint64_t* credit_in, void* k_out,
                               void* v_out, uint64_t* credit_out, int32_t* kept_out,
                               float* u_out, void* stream);

/* ---------------------------------------------------------------------------
 * 8-bit paged cache: the compacted (or whole) cache held as 8-bit codes with
 * one fp32 scale for each (page, KV head), in the pages of kvc_gather_paged.
 * The value of a code is code * scale of its page and head.
 *   KVC_Q8_E4M3  codes are OCP e4m3 (4 significant bits, largest value 448);
 *                kvc_q8_store and kvc_q8_append give a page the smallest
 *                scale 2^e, e >= -126, with max|x| <= 448 * 2^e: coding again
 *                under a larger scale only shifts exponents
 *   KVC_Q8_INT8  codes -127..127; scale = max(max|x| / 127, 2^-126) and
 *                code = rint(x * (1 / scale)), both in fp32
 * kvc_q8_load and kvc_q8_attend take any finite non-negative scale.
 *
 * Layout: k_pool, v_pool 8-bit [n_blocks][kv_heads][block_size][head_dim]
 * (16-byte aligned), k_scale, v_scale f32 [n_blocks][kv_heads], table i32
 * [n_seqs][table_blocks], seq_len i32 [n_seqs] (device arrays).  Head n =
 * b * kv_heads + h of the bf16 arrays is head h of sequence b; its position
 * t lives in page table[b][t / block_size], row t % block_size.  A table
 * entry outside [0, n_blocks) names no page: its positions are not attended,
 * load as zeros and are not written.  seq_len is taken as clamped to [0, cap]
 * with cap = min(max_len, table_blocks * block_size) (max_len 0: the second).
 * Rows of a page at or past seq_len are neither read nor written; their codes
 * may be anything.  Preconditions (not checked): the codes of attended
 * positions are finite, and a page that is written belongs to one entry of
 * the table. */
typedef struct kvc_q8_cache {
  int32_t n_seqs;        /* B sequences; 0 = nothing to do                   */
  int32_t kv_heads;      /* H KV heads, n_seqs * kv_heads < 2^24             */
  int32_t head_dim;      /* d, 64 or 128                                     */
  int32_t block_size;    /* positions per page, 1..4096                      */
  int32_t table_blocks;  /* table entries per sequence (>= 1),
                            table_blocks * block_size <= 2^30                */
  int32_t max_len;       /* 0, or a bound on seq_len that sizes the launches */
  int32_t format;        /* KVC_Q8_E4M3 or KVC_Q8_INT8                       */
  int32_t reserved;      /* 0                                                */
  int64_t n_blocks;      /* pages in the pools, n_blocks * kv_heads *
                            block_size < 2^32 - 1                            */
  void* k_pool;
  void* v_pool;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  const int32_t* seq_len;
} kvc_q8_cache;

/* Step 5 into 8-bit pages: writes slots 0..L-1 of every sequence and the
 * scales of their pages.  k, v: bf16 [n_seqs * kv_heads][t_stride][d], rows
 * 0..T-1 valid, T 1..2^27.  With kept (i32 [n_seqs * kv_heads][n_kept], as the event
 * writes it) slot j of head n is row kept[n][j] (zeros where it is outside
 * [0, T)) and L = min(seq_len, n_kept); kept NULL (n_kept 0) stores the last L
 * = min(seq_len, T) rows: slot j is row T - L + j, the left-padded layout of
 * kvc_params.valid_len.  A page's scale covers the slots written to it; rows
 * past L in the last page are left as they were.  Heads times the pages that
 * min(T or n_kept, cap) slots fill, K and V counted, at most 2^32 - 256.
 * Precondition: the rows are finite.  No workspace. */
int kvc_q8_store(const kvc_q8_cache* c, int32_t T, int32_t t_stride, const int32_t* kept,
                 int32_t n_kept, const void* k, const void* v, void* stream);

/* The cache as bf16 rows, for the event's scores or to move it: row T - L + t
 * of k_out, v_out (bf16 [n_seqs * kv_heads][t_stride][d]) receives position t,
 * L = seq_len, for the last min(L, T) positions; rows 0..T-L-1 are zeros
 * (left padding), rows >= T untouched; T 1..2^27.  Each value is code * scale in fp32,
 * rounded once.  k_out or v_out may be NULL (not loaded).  No workspace. */
int kvc_q8_load(const kvc_q8_cache* c, int32_t T, int32_t t_stride, void* k_out, void* v_out,
                void* stream);

/* Appends: the last `window` positions of every sequence (seq_len counts them
 * already) receive k_new, v_new (bf16 [n_seqs * kv_heads][window][d]); new row
 * w goes to position seq_len - window + w (skipped where negative).  n_new: NULL,
 * or i32 [n_seqs] on the device: sequence b appends its last n_new[b] rows only
 * (clamped to 0..window), the rows before them are skipped.  A page
 * whose first row is new takes its scale from the new rows.  One that holds
 * earlier rows keeps its scale unless the new rows alone need a larger one;
 * then its earlier rows are coded again under the larger scale (e4m3: code *
 * old / new rounded to nearest even; int8: rint(code * (old * (1 / new)))).
 * The same call repeated changes nothing.  Heads times the pages that window
 * positions can touch: at most 2^32 - 256.  Precondition: the rows are finite.
 * No workspace. */
int kvc_q8_append(const kvc_q8_cache* c, int32_t window, const int32_t* n_new, const void* k_new,
                  const void* v_new, void* stream);

/* Attention of the last `window` positions' queries over the cache.  q, out:
 * bf16 [n_seqs * kv_heads][group][window][d] (the layout of q_win); query w
 * sits at position seq_len - window + w and attends to the positions up to
 * its own:  out = sum_t softmax_t(scale * <q, k[t]>) * v[t], in fp32, lse:
 * optional f32 [n_seqs * kv_heads][group][window], log(sum_t exp(scale *
 * <q, k[t]>)).  scale 0 => 1/sqrt(d), otherwise positive, at most 2^127.  A query
 * that attends to nothing gives zeros and lse = -inf.  Held in fewer bits: a
 * query element below 2^-29 of its row's largest loses some; a key's weight *
 * value scale enters the product with the codes as fp16, 11 bits down to 2^-23 of
 * the row's largest and within 2^-34 of that largest below (the sum of the weights
 * is fp32); a value scale more than 2^100 below the largest among the same piece
 * of at most 2048 keys, attended to or not, counts as 2^-100 of it, too large
 * where a query attends to nothing louder.  Otherwise keys that a query does not
 * attend to change its roundings at most.
 * group 1..64, window >= 1, group * window <= 4096.
 * A head's results depend on its own length, queries and pages alone.
 * ws: at least kvc_q8_attend_workspace_bytes(c, group, window), 256-byte
 * aligned (may be NULL when that is 0). */
int kvc_q8_attend(const kvc_q8_cache* c, int32_t group, int32_t window, float scale,
                  const void* q, void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes kvc_q8_attend needs; (size_t)-1 for invalid arguments (the
 * device pointers are not looked at).  Pure host function. */
size_t kvc_q8_attend_workspace_bytes(const kvc_q8_cache* c, int32_t group, int32_t window);

/* ---------------------------------------------------------------------------
 * Pages: who owns which page of a pool, kept on the device.  refs[p] counts
 * the table entries that name page p; a page with refs <= 0 is free.  A new
 * page is always the lowest free one, so the same calls give the same tables.
 * The calls change table, seq_len and refs in place (kvc_pages_compact writes
 * new ones); table entries outside [0, n_blocks) name no page.  Precondition
 * (not checked): refs agrees with the tables of all its users.
 * Requests that need new pages are served in order; from the first that does
 * not fit on, none gets a page.  status (i32, device): 0 served, 1 no room,
 * 2 refused; a request with status 1 or 2 changed nothing. */
typedef struct kvc_page_table {
  int32_t n_seqs;        /* sequences, 0..2^20 (0 = nothing to allocate or
                            free; forks and compactions need at least one)   */
  int32_t table_blocks;  /* entries per sequence (>= 1), table_blocks *
                            block_size <= 2^30                               */
  int32_t block_size;    /* positions per page, 1..4096                      */
  int32_t n_blocks;      /* pages in the pool, 1..2^24                       */
  int32_t* table;        /* i32 [n_seqs][table_blocks]                       */
  int32_t* seq_len;      /* i32 [n_seqs]                                     */
  int32_t* refs;         /* i32 [n_blocks]                                   */
} kvc_page_table;

/* An array indexed by page: page p is the page_bytes bytes at base + p *
 * page_bytes (a pool, bf16 or 8-bit, or the scales of one). */
typedef struct kvc_page_buffer {
  void* base;
  int64_t page_bytes;
} kvc_page_buffer;

/* Gives every sequence b pages for its positions 0..want_len[b]-1: entries
 * among its first ceil(want_len[b] / block_size) that name no page receive
 * one, all or none per sequence.  want_len: i32 [n_seqs], 0 = leave alone,
 * negative or past the table: status 2.  seq_len is not changed (want_len may be
 * seq_len itself).
 * status: i32 [n_seqs]. */
int kvc_pages_alloc(const kvc_page_table* t, const int32_t* want_len, int32_t* status, void* ws,
                    size_t ws_bytes, void* stream);

/* Forks: for each pair i, sequence dst[i] gives up the pages it holds and
 * becomes a copy of src[i]: it shares the floor(len / block_size) full pages,
 * and an open last page is copied to a new page in all n_bufs buffers (host
 * array; n_bufs 0..4096).  Pages given up are free from the next call on.
 * What a sequence appends to is then its own; one that is cut back into a page
 * it shares (a shorter seq_len) has to be forked again before it appends.
 * src, dst: i32 [n_pairs] on the device.  Status 2: an id out of range, src
 * = dst, dst named by an earlier pair, or src named as dst by any pair.
 * status: i32 [n_pairs]. */
int kvc_pages_fork(const kvc_page_table* t, int32_t n_pairs, const int32_t* src,
                   const int32_t* dst, const kvc_page_buffer* bufs, int32_t n_bufs,
                   int32_t* status, void* ws, size_t ws_bytes, void* stream);

/* Frees the sequences ids[0..n_ids-1] (i32 on the device; out of range:
 * skipped, named twice: freed once): their pages lose one count each, their
 * entries become -1, their lengths 0.  No workspace. */
int kvc_pages_free(const kvc_page_table* t, int32_t n_ids, const int32_t* ids, void* stream);

/* Copies page src[i] to page dst[i] in every buffer, i < n_pairs (i32 on the
 * device; a pair with an id outside [0, n_blocks) is skipped).  Precondition:
 * the destinations are distinct and none of them is a source.  No
 * workspace. */
int kvc_pages_copy(int32_t n_blocks, int32_t n_pairs, const int32_t* src, const int32_t* dst,
                   const kvc_page_buffer* bufs, int32_t n_bufs, void* stream);

/* Compacts the pool: with n_live pages in use, those at or past n_live move,
 * in ascending order, to the free pages below it, in all buffers.  table_out
 * (i32 [n_seqs][table_blocks]) and refs_out (i32 [n_blocks]) receive the new
 * tables and counts, remap (i32 [n_blocks]) the new id of every page (-1: it
 * was free), n_live (i32 [1]) the count; t's own arrays are read only, and
 * swapping them is the caller's.  Other tables that name these pages follow by
 * remap. */
int kvc_pages_compact(const kvc_page_table* t, const kvc_page_buffer* bufs, int32_t n_bufs,
                      int32_t* table_out, int32_t* refs_out, int32_t* remap, int32_t* n_live,
                      void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes kvc_pages_alloc, kvc_pages_fork (with up to n_pairs pairs)
 * and kvc_pages_compact need; 0 for invalid arguments.  Pure host function. */
size_t kvc_pages_workspace_bytes(const kvc_page_table* t, int32_t n_pairs);

/* Workspace bytes any entry point that takes a kvc_params needs for these parameters (0 when
 * the parameters are invalid).  Pure host function. */
size_t kvc_workspace_bytes(const kvc_params* p);

/* Segment capacity S per head: n_cut + 1 + floor(T/seg_max) capped at T,
 * with n_cut = #{k >= 1 : k*delta < 1} (or ceil(T/seg_fixed) - 1 with fixed
 * segments); seg_max = 0 drops the second term.  Returns a negative status
 * for invalid parameters.  Pure host function. */
int kvc_segment_capacity(const kvc_params* p);

/* Validates the parameters alone (no pointers): KVC_OK or the error code.
 * Pure host function. */
int kvc_check_params(const kvc_params* p);

/* Static description of a status code. */
const char* kvc_strerror(int status);

/* KVC_ABI_VERSION of the built library. */
int kvc_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVC_H */
