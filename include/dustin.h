/*
 * dustin.h -- C-ABI of the GB300 (sm_103a) library for Dustin's
 * draft-augmented sparse verification hot path.
 *
 * Sources of the operations (cited by page title and section):
 *   [Paper]  "Dustin: Draft-Augmented Sparse Verification for Efficient
 *            Long-Context Generation with Speculative Decoding"
 *            (arXiv 2606.24957, HTML translation), section 3.1 Eq. (1)-(4).
 *   [Notes]  "dustin-long-context" paper notes: section 2.2 (S_Draft,
 *            S_Target, one global index set, Fig. 5), section 2.3
 *            (I_verify = sink + window + draft top-m + target rest),
 *            section 2.4 (SRH: scoring on a few (layer, head) pairs, Fig. 6),
 *            section 3 (Fig. 7 self-attention speedup against full cache).
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library keeps no reference after the call returns and allocates
 *     no device memory.  Scratch space, where a call needs it, is passed by
 *     the caller as (ws, ws_bytes), sized by the matching *_workspace_size
 *     query for the current device.
 *   - bf16 tensors are IEEE bfloat16 bit patterns (uint16), row-major, with
 *     the innermost (head-dim) axis contiguous.  Base pointers and row
 *     strides must be 16-byte aligned.
 *   - Every compute call is asynchronous on `stream` (a cudaStream_t; NULL
 *     is the legacy default stream) and returns a dustin_status.  Arguments
 *     are validated on the host before anything is launched: an invalid call
 *     launches nothing.  A failed launch returns DUSTIN_ERR_CUDA with the
 *     CUDA error text in dustin_last_error().  Nothing is thrown across the
 *     ABI and no kernel traps.
 *   - Device-side checks (an index >= n, a page id outside the pool) never
 *     fault: the offending position is left out of the attention and a flag
 *     is raised, read with dustin_device_status().  Every wait inside a
 *     kernel is bounded (about one second); one that gives up raises
 *     DUSTIN_DEVFLAG_WAIT_TIMEOUT and the kernel returns.
 *   - Grouped-query attention: query head h reads kv head h / (h_q / h_kv).
 */
#ifndef DUSTIN_H_
#define DUSTIN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dustin_status {
  DUSTIN_OK = 0,
  DUSTIN_ERR_INVALID_ARG = 1, /* NULL pointer where one is needed, bad enum */
  DUSTIN_ERR_SHAPE = 2,       /* sizes inconsistent or out of range         */
  DUSTIN_ERR_UNSUPPORTED = 3, /* valid but not built (e.g. d not 64 / 128)  */
  DUSTIN_ERR_WORKSPACE = 4,   /* workspace NULL or smaller than required    */
  DUSTIN_ERR_ALIGNMENT = 5,   /* pointer or stride not 16-byte aligned      */
  DUSTIN_ERR_CUDA = 6,        /* a CUDA runtime call failed                 */
  DUSTIN_ERR_DEVICE = 7       /* a device-side check raised a flag          */
} dustin_status;

/* Device-side flags reported by dustin_device_status(). */
#define DUSTIN_DEVFLAG_INDEX_RANGE 0x1u /* idx[b][i] < 0 or >= n            */
#define DUSTIN_DEVFLAG_PAGE_RANGE 0x2u  /* page id < 0 or >= num_pages      */
#define DUSTIN_DEVFLAG_WAIT_TIMEOUT 0x4u /* a pipeline wait gave up (~1 s);
                                            the outputs of that call are void */
#define DUSTIN_DEVFLAG_NO_PAGES 0x8u     /* a sequence could not grow        */
#define DUSTIN_DEVFLAG_INDEX_ORDER 0x10u /* compaction in place over indices
                                            that do not ascend strictly      */

#define DUSTIN_NORM_NONE 0 /* hybrid mix of the raw score vectors          */
#define DUSTIN_NORM_L1 1   /* each score vector divided by its own sum     */

#define DUSTIN_DTYPE_F32 0  /* IEEE binary32                                */
#define DUSTIN_DTYPE_BF16 1 /* bfloat16 bit patterns                        */

/*
 * One layer's KV cache for one (layer) of the target or the draft.
 *
 * Contiguous layout (page_table == NULL): element (b, kv head h, position
 * j, dim c) is at  base + b*stride_b + h*stride_h + j*stride_n + c.
 * Paged layout (page_table != NULL): a pool of pages [page][h_kv][page_size]
 * [d]; position j of sequence b lives in page
 * p = page_table[b*pages_per_seq + j/page_size] at
 * base + p*stride_b + h*stride_h + (j % page_size)*stride_n + c, so stride_b
 * is then the stride between pages.  page_table is a device int32 array.
 * page_size is a positive multiple of 16 (scoring reads pages of 16, 32 or
 * 64 positions as one TMA box each; other sizes take a cp.async path).
 * v may be NULL for calls that read keys only (scoring).
 * Strides are in elements; every stride must be a multiple of 8 (16 bytes).
 */
typedef struct dustin_kv {
  const void* k;
  const void* v;
  int64_t stride_b;
  int64_t stride_h;
  int64_t stride_n;
  const int32_t* page_table;
  int32_t page_size;
  int32_t pages_per_seq;
  int32_t num_pages;
} dustin_kv;

/* Text for a status code (static storage, never NULL). */
const char* dustin_status_string(int status);

/* Detail of the last failing call on this host thread ("" if none). */
const char* dustin_last_error(void);

/* Library ABI version: major*10000 + minor*100 + patch. */
int dustin_version(void);

/* Number of kernels this library has launched in this process. */
uint64_t dustin_launch_count(void);

/*
 * Reads and clears the device-side flags (DUSTIN_DEVFLAG_*) of the current
 * device.  Synchronises the device.  Returns DUSTIN_ERR_DEVICE if any flag
 * was set, DUSTIN_OK otherwise; *flags (may be NULL) receives the flags.
 */
int dustin_device_status(uint32_t* flags);

/*
 * Self-test of the bounded wait that every pipeline wait of the library
 * uses: launches one CTA of 32 threads on `stream` that waits on an
 * mbarrier no thread ever arrives at, with a limit of `limit_cycles` SM
 * clock cycles (1 .. 2^31; about 2 * 10^9 inside the compute calls).  The
 * wait gives up, raises DUSTIN_DEVFLAG_WAIT_TIMEOUT and the kernel returns:
 * the context stays usable.  Returns DUSTIN_ERR_SHAPE for a limit outside
 * that range, DUSTIN_ERR_CUDA if the launch fails, DUSTIN_OK otherwise.
 */
int dustin_wait_selftest(int64_t limit_cycles, void* stream);

/* ------------------------------------------------------------------------
 * Importance scoring on the scored (layer, head) pairs.
 *
 * [Notes] section 2.2: S_Draft sums the draft's attention over its heads,
 * layers and Gamma lookahead queries; S_Target sums the target's attention
 * of its latest token over its heads and layers.  [Notes] section 2.4
 * (Fig. 6): only the selected (layer, head) pairs are recomputed.
 *
 *   s_out[b][j] = sum_{p < n_pairs} sum_{r < rows}
 *                 softmax_j( scale * q[p][b][r] . K_p[b][kv_head[p]][j] )
 * over history positions j in [0, n); fp32 out, fp32 accumulation.
 *
 *   q        bf16 [n_pairs][b][rows][d], device
 *   kv       host array [n_pairs]: the key cache of pair p's layer (v unused)
 *   kv_head  host array [n_pairs]: kv head of pair p (q_head / group)
 *   s_out    fp32 [b][n], device, fully overwritten
 *   ws       device scratch of dustin_score_heads_workspace_size() bytes
 * Called once for the target (rows = 1) and once for the draft
 * (rows = Gamma).  Limits: d in {64, 128}; 1 <= rows <= 16;
 * 1 <= n_pairs <= 64; n_pairs * rows <= 1024.
 * b == 0 or n == 0 is a no-op.
 */
size_t dustin_score_heads_workspace_size(int b, int n, int n_pairs, int rows);
int dustin_score_heads(int b, int n, int d, int n_pairs, int rows,
                       const void* q, const dustin_kv* kv,
                       const int32_t* kv_head, float scale, float* s_out,
                       void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Scoring without a caller-provided workspace.  The paper has no
 * counterpart: this is a convenience of this library.
 *
 * For callers that cannot allocate device memory when they score -- for
 * example a serving loop that has given all of HBM to the KV cache (a
 * cudaMalloc there fails or stalls the step), or a plugin whose framework
 * owns the allocator and hands over only inputs and outputs.  Same inputs,
 * outputs and limits as dustin_score_heads, but the scratch lives in a fixed
 * array of DUSTIN_NOALLOC_SCRATCH_BYTES compiled into the library (every GPU
 * that loads the library keeps it until the process exits).  The call
 * allocates nothing.
 *   - A call whose scratch (dustin_score_heads_workspace_size) exceeds the
 *     array is rejected with DUSTIN_ERR_WORKSPACE before anything runs.
 *   - The argument checks of dustin_score_heads run first (same statuses);
 *     then a call whose scratch (dustin_score_heads_workspace_size) exceeds
 *     the array is rejected with DUSTIN_ERR_WORKSPACE before anything runs.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.  The address is remembered per device and
 *     CUDA context: after cudaDeviceReset the next call looks it up again
 *     (again outside any capture).
 *   - All calls share the one array, which keeps the last call's contents.
 *     Each call overwrites every scratch byte it reads, so nothing needs
 *     clearing, but calls that overlap on the GPU (other streams, other
 *     threads) race on the array: serialise them.
 */
#define DUSTIN_NOALLOC_SCRATCH_BYTES (64u << 20)
int dustin_score_heads_noalloc(int b, int n, int d, int n_pairs, int rows,
                               const void* q, const dustin_kv* kv,
                               const int32_t* kv_head, float scale,
                               float* s_out, void* stream);
/* Size in bytes of that built-in array (DUSTIN_NOALLOC_SCRATCH_BYTES of the
 * library as built), for callers that plan around it at run time. */
size_t dustin_score_heads_noalloc_capacity(void);

/* ------------------------------------------------------------------------
 * Hybrid combination and global per-sequence Top-K ([Notes] sections 2.2
 * and 2.3).  One index set per sequence, shared by all layers and heads.
 *
 * Protected positions [0, n_sink) and [n - n_recent, n) are always kept;
 * k counts them.  The remaining budget r = k - |protected| is filled from
 * the other positions:
 *   m < 0  (alpha mode): top-r of c_j = a_D*S_D[j] + a_T*S_T[j], where
 *          a_D = alpha / sum(S_D) and a_T = (1 - alpha) / sum(S_T) under
 *          DUSTIN_NORM_L1 (alpha and 1 - alpha under DUSTIN_NORM_NONE).
 *          Sums in fp64, coefficients rounded once to fp32, then
 *          c_j = fl(fl(a_D*S_D[j]) + fl(a_T*S_T[j])) in fp32 round-to-nearest.
 *          A term with weight 0 or a NULL vector is left out.  A sum that is
 *          not positive and finite leaves that vector unscaled.
 *   m >= 0 (budget split): top-min(m, r) of S_D, then the top of S_T for the
 *          rest of the budget over the positions not yet taken.
 * Order: higher score first, ties to the lower position; -0 equals +0; NaN
 * ranks below every number.  idx rows come out strictly ascending.
 * k >= n keeps all n positions (idx row length n).
 *
 *   s_draft, s_target  fp32 [b][n], device; either may be NULL (not both)
 *   idx                int32 [b][min(k, n)], device, fully overwritten
 * Errors: |protected| > k with k < n is DUSTIN_ERR_SHAPE.  n <= 2^20.
 */
int dustin_hybrid_topk(int b, int n, int k, int n_sink, int n_recent,
                       double alpha, int m, int norm, const float* s_draft,
                       const float* s_target, int32_t* idx, void* stream);

/* ------------------------------------------------------------------------
 * Sparse verification attention ([Notes] section 2.2 Fig. 5, Stage 2: the
 * target verifies its w window rows over the selected KV only).
 *
 * For each sequence b, query head h and window row t (no causal mask: all
 * selected history precedes the window; the window's own causal block is
 * merged by the caller through lse):
 *   o[b][h][t]   = softmax_i(scale * q[b][h][t] . K[b][g][idx[b][i]]) V[..]
 *   lse[b][h][t] = log sum_i exp(scale * q[b][h][t] . K[b][g][idx[b][i]])
 * with g = h / (h_q / h_kv).  k == 0 gives o = 0, lse = -inf.
 *
 *   q    bf16 [b][h_q][w][d], device (contiguous)
 *   kv   host pointer to one dustin_kv (k and v both required)
 *   idx  int32 [b][k], device, each entry in [0, n); ascending order is
 *        fastest but not required
 *   o    bf16 [b][h_q][w][d], device;  lse fp32 [b][h_q][w] (natural log)
 *   ws   device scratch of dustin_sparse_verify_attn_workspace_size() bytes
 *        (may be 0 bytes; ws may then be NULL)
 *   flags  0, or DUSTIN_ATTN_KV_READY (below)
 * Limits: d in {64, 128}; h_q a multiple of h_kv; k <= n; scale finite and
 * > 0; flags has no other bit set (DUSTIN_ERR_INVALID_ARG).
 */
size_t dustin_sparse_verify_attn_workspace_size(int b, int h_q, int h_kv,
                                                int d, int w, int k);
int dustin_sparse_verify_attn(int b, int h_q, int h_kv, int d, int w, int n,
                              int k, const void* q, const dustin_kv* kv,
                              const int32_t* idx, float scale, void* o,
                              float* lse, void* ws, size_t ws_bytes,
                              unsigned flags, void* stream);

/* The same with the window's own causal block merged in (the w window
 * tokens follow the history, so window row t also attends to window
 * positions 0..t, as in ordinary causal decoding):
 *   o[b][h][t] = softmax over [idx[b][0..k), window 0..t] of scale * q . K
 *   lse        = log sum exp over the same positions
 * where the window part reads win (k and v both required, contiguous, no
 * page table): bf16 [b][h_kv][w][d] through win->stride_b/h/n.  Same
 * workspace as dustin_sparse_verify_attn.  With DUSTIN_ATTN_KV_READY the
 * window rows, like q, are read only after the preceding kernel finished.
 * (The sparse call's LSE lets a caller merge this block itself; this entry
 * point does it inside the same launch, as one more tile of w rows.) */
int dustin_sparse_verify_attn_window(int b, int h_q, int h_kv, int d, int w,
                                     int n, int k, const void* q,
                                     const dustin_kv* kv, const int32_t* idx,
                                     const dustin_kv* win, float scale, void* o,
                                     float* lse, void* ws, size_t ws_bytes,
                                     unsigned flags, void* stream);

/* Sparse verification attention of n_layers layers in one persistent
 * launch: for each layer l, the call dustin_sparse_verify_attn(b, h_q, h_kv,
 * d, w, n, k, q[l], &kv[l], idx, scale, o[l], lse[l]) with one index set
 * for all layers.  For callers that hold several layers' queries at once
 * (the layers of one model run one after another, so within a single
 * forward pass only one layer is ready at a time).  The (layer, sequence,
 * kv head, row block) units are dealt round-robin to one CTA per SM, which
 * streams them back to back without draining its pipeline.
 *   q, o, lse  host arrays [n_layers] of device pointers (as in the sparse
 *              call); kv host array [n_layers] of descriptors, all paged or
 *              all contiguous
 *   flags      0 or DUSTIN_ATTN_KV_READY (accepted, no effect)
 * No workspace.  Limits as the sparse call, and k <= 2048
 * (DUSTIN_ERR_UNSUPPORTED); any number of layers (launches of up to 128).
 * Not an API of the paper. */
int dustin_sparse_verify_attn_layers(int n_layers, int b, int h_q, int h_kv, int d,
                                     int w, int n, int k, const void* const* q,
                                     const dustin_kv* kv, const int32_t* idx,
                                     float scale, void* const* o, float* const* lse,
                                     unsigned flags, void* stream);

/* ------------------------------------------------------------------------
 * Quest page scoring: the page-level baseline selector of the comparison
 * ([Notes] section 1 and related work; "Quest-16" in Fig. 8).  Not part of
 * Dustin; for measurements beside it.
 *
 * dustin_quest_page_stats: per page of `page` consecutive positions (the
 * last may be short), the channel-wise minimum and maximum of the keys:
 *   stats bf16 [b][h_kv][P][2][d], P = ceil(n / page), minimum row first;
 *   dustin_quest_stats_size() bytes, 16-byte aligned.
 * kv: keys only (v unused), contiguous or paged.  In Quest the statistics
 * are kept up to date as tokens are appended, not rebuilt every step.
 *
 * dustin_quest_page_scores: for one query row per head, q bf16 [b][h_q][d],
 *   scores[b][h][p] = sum_c max(q[b][h][c] * min_c, q[b][h][c] * max_c)
 * with the stats of kv head h / (h_q / h_kv): the largest q . k over the
 * page's channel box.  scores fp32 [b][h_q][P].  The top pages per (b, h)
 * come from dustin_hybrid_topk on scores viewed as b*h_q rows of P (alpha
 * 1, s_target NULL, norm NONE, no protected positions).
 * At most 64 query heads per kv head. */
size_t dustin_quest_stats_size(int b, int h_kv, int d, int n, int page);
int dustin_quest_page_stats(int b, int h_kv, int d, int n, int page,
                            const dustin_kv* kv, void* stats, void* stream);
int dustin_quest_page_scores(int b, int h_q, int h_kv, int d, int n, int page,
                             const void* q, const void* stats, float* scores,
                             void* stream);

/* DUSTIN_ATTN_KV_READY: the caller guarantees that idx, the page table and
 * the K/V cache were complete before the kernel enqueued just before this
 * call on `stream` started (that kernel does not write them; q may be its
 * output).  The attention kernels are launched with programmatic dependent
 * launch and may then gather their first K/V tiles while that kernel is
 * still running; q is read, and o, lse and ws are written, only after it
 * has finished.  This holds, for example, for consecutive layers'
 * verification attention over one index set whose K/V were appended
 * before the step.  Without the flag nothing is read early.  A wrong
 * promise gives stale rows, never a fault.  Not an API of the paper: a
 * launch-overlap hint. */
#define DUSTIN_ATTN_KV_READY 1u

/* ------------------------------------------------------------------------
 * Full-cache verification attention: the dense in-run baseline ([Notes]
 * section 3, Fig. 7 "Full Cache").  The sparse call over idx = 0..n-1;
 * flags as there (DUSTIN_ATTN_KV_READY: the page table and K/V).
 */
size_t dustin_full_verify_attn_workspace_size(int b, int h_q, int h_kv,
                                              int d, int w, int n);
int dustin_full_verify_attn(int b, int h_q, int h_kv, int d, int w, int n,
                            const void* q, const dustin_kv* kv, float scale,
                            void* o, float* lse, void* ws, size_t ws_bytes,
                            unsigned flags, void* stream);
/* The full-cache call with the window's causal block merged in, as
 * dustin_sparse_verify_attn_window.  dustin_full_verify_attn_workspace_size
 * covers both. */
int dustin_full_verify_attn_window(int b, int h_q, int h_kv, int d, int w, int n,
                                   const void* q, const dustin_kv* kv,
                                   const dustin_kv* win, float scale, void* o,
                                   float* lse, void* ws, size_t ws_bytes,
                                   unsigned flags, void* stream);

/* ------------------------------------------------------------------------
 * Verification attention of a batch whose sequences share prefixes (samples
 * of one prompt, requests under one system prompt).  Not an API of the
 * paper.  The b sequences form `groups` groups of b / groups consecutive
 * ones; group g's sequences share the P_g positions of row g of `prefix`,
 * and sequence i goes on with the L_i positions of row i of `own` and, with
 * win, the w window positions (causal, as in the *_window calls):
 *   o[i][h][t] = softmax over [prefix g 0..P_g), own 0..L_i), window 0..t]
 *                of scale * q . K, times V;   lse = log sum exp (natural)
 * for g = i / (b / groups).  The prefix is read once per kv head and row
 * tile of 256 query rows, not once per sequence.  A row that sees no
 * position, or only scores of -inf, gives o = 0, lse = -inf.  A row with a
 * score that is NaN or +inf gives NaN, o and lse.
 *
 *   q           bf16 [b][h_q][w][d], device (contiguous); o like q; lse fp32
 *               [b][h_q][w]
 *   prefix      one row (contiguous cache or page-table row) per group;
 *               ignored (may be NULL) if n_prefix is 0
 *   prefix_len  int32 [groups], device, or NULL (n_prefix each); own_len
 *               int32 [b] or NULL (n_own each); clamped to [0, n_prefix],
 *               [0, n_own]
 *   own         one row per sequence; ignored if n_own is 0.  Where a fork
 *               shares whole pages, a sequence's own positions are the rest
 *               of its page-table row: page_table + shared pages, with the
 *               full row's pages_per_seq
 *   win         [b][h_kv][w][d], contiguous, or NULL
 * Positions behind the lengths are never used, whatever they hold; window
 * rows, however, are weighted with exact zeros above the diagonal, so V of
 * the window is finite.  Pages outside the pool are left out
 * (DUSTIN_DEVFLAG_PAGE_RANGE).  DUSTIN_ATTN_KV_READY is accepted, without
 * effect.  Sums are taken in a fixed order: equal calls give equal bits.
 * Precision: scores, maxima, sums and partial results are fp32, but a weight is
 * rounded to bf16 for its product with V (the sum it is divided by is of the
 * unrounded ones), and o once more: o is off by up to 2^-8 (sum_j p_j |V_j| +
 * |o|), element by element, beside fp32 rounding; lse by fp32 rounding alone.
 * Limits: as dustin_sparse_verify_attn; kv strides below 2^39 elements; b <=
 * 2^20; n_prefix, n_own <= 2^27; 2^23 products of 128 rows with 128 positions
 * in all; a workspace of 2^35 bytes.  Beyond them: DUSTIN_ERR_SHAPE.
 * Workspace: dustin_prefix_verify_attn_workspace_size (with or without win);
 * its content need not be kept, and calls that may run at the same time (two
 * streams, two captured graphs) have one each.
 */
size_t dustin_prefix_verify_attn_workspace_size(int b, int groups, int h_q, int h_kv,
                                                int d, int w, int n_prefix, int n_own);
int dustin_prefix_verify_attn(int b, int groups, int h_q, int h_kv, int d, int w,
                              int n_prefix, int n_own, const void* q,
                              const dustin_kv* prefix, const int32_t* prefix_len,
                              const dustin_kv* own, const int32_t* own_len,
                              const dustin_kv* win, float scale, void* o, float* lse,
                              void* ws, size_t ws_bytes, unsigned flags, void* stream);

/* ------------------------------------------------------------------------
 * Verification of drafted tokens (speculative sampling), the step that
 * follows the target's pass over its w verification rows.  Not an API of the
 * paper.
 *
 * Sequence i has g = n_draft[i] drafted tokens x_0 .. x_{g-1} (g <= w - 1;
 * n_draft NULL: w - 1 each; values outside [0, w - 1] are clamped), the
 * draft model's distribution q_t over the vocabulary each was drawn from,
 * and the target's distributions p_0 .. p_g.  Draft t is accepted while
 *   u_accept[i][t] * q_t(x_t) < p_t(x_t)      (products compared exactly),
 * up to the first that is not.  With a drafts accepted, one more token is
 * drawn by inversion: the first j with C_j > u_sample[i] * C_last, where C
 * is the running sum, over ascending tokens, of
 *   max(p_a(j) - q_a(j), 0)   if a < g (a draft was rejected),
 *   p_a(j)                    if a == g, or if that residual has no mass.
 * So the tokens follow the target's distribution if u_accept and u_sample
 * are independent uniforms in [0, 1).  With p_draft NULL the drafts are
 * taken as certain (q is 1 at the draft, 0 elsewhere), as for drafts found
 * by lookup.  Entries that are negative, NaN or infinite have no mass: they
 * count as 0, in the acceptance too, so no u_accept >= 0 accepts a draft
 * without mass in the target's row.  The sums carry about 48 bits (a row's
 * masses add up to less than 2^127, as probabilities do).  u_sample <= 0 or
 * NaN counts as 0, >= 1 as the last token with mass; a NaN in u_accept
 * rejects.  A draft outside
 * [0, vocab) is rejected and raises DUSTIN_DEVFLAG_INDEX_RANGE.
 *
 *   p_target   [b][w][vocab] of `dtype` (DUSTIN_DTYPE_*), device; row (i, t)
 *              at element i*stride_tb + t*stride_tw, entries contiguous
 *   p_draft    [b][w-1][vocab] of the same type, row strides stride_db,
 *              stride_dw; may be NULL
 *   draft      int32 [b][w-1];  n_draft int32 [b] or NULL
 *   u_accept   fp32 [b][w-1];   u_sample fp32 [b]
 *   tokens     int32 [b][w]: the a accepted drafts, the drawn token (-1 if
 *              the target's row has no mass at all), then -1
 *   n_accepted int32 [b]: a
 * draft and u_accept may be NULL when w == 1.  Rows may start at any
 * element; they are read in aligned words of 16 bytes, so bytes beside a row
 * may be read too (never used).
 * b == 0 is a no-op.  Limits: vocab >= 1, b <= 2^27.  No workspace. */
int dustin_verify_tokens(int b, int w, int vocab, int dtype, const void* p_target,
                         int64_t stride_tb, int64_t stride_tw, const void* p_draft,
                         int64_t stride_db, int64_t stride_dw, const int32_t* draft,
                         const int32_t* n_draft, const float* u_accept,
                         const float* u_sample, int32_t* tokens, int32_t* n_accepted,
                         void* stream);

/* ------------------------------------------------------------------------
 * Compaction of a KV cache to an index set (for example the one of
 * dustin_hybrid_topk, or the accepted path of a token tree): for every
 * layer l, kv head and i < k_len[b],
 *   row i of sequence b in dst[l] = row idx[b][i] of sequence b in src[l],
 * K and V.  Rows from k_len[b] on are left as they were.
 *
 *   src, dst  host arrays [n_layers]; contiguous or paged, each on its own
 *             (all layers of a side alike); src holds n positions, dst at
 *             least k
 *   idx       int32 [b][k], device; entries outside [0, n) raise
 *             DUSTIN_DEVFLAG_INDEX_RANGE and leave their row as it was, and
 *             so do pages outside the pool (DUSTIN_DEVFLAG_PAGE_RANGE)
 *   k_len     int32 [b], device, or NULL (k each); clamped to [0, k]
 * In place (dst[l] and src[l] have the same base and page table) the
 * entries of a row ascend strictly; rows that stay where they are are not
 * written (so a shared prefix that is kept whole may lie on shared pages).
 * Otherwise (DUSTIN_DEVFLAG_INDEX_ORDER) that sequence's rows are
 * unspecified.  Out of place, src and dst rows must not overlap, and an
 * index may repeat.  Rows of dst are distinct: a stride of 0 is refused, two
 * sequences' rows on one page are the caller's to avoid.  Limits: d in {64,
 * 128}; k <= n in place; k <= 2^30; b * h_kv * min(n_layers, 128) <= 2^24. */
int dustin_kv_compact(int n_layers, int b, int h_kv, int d, int n, int k,
                      const dustin_kv* src, const dustin_kv* dst, const int32_t* idx,
                      const int32_t* k_len, void* stream);

/* ------------------------------------------------------------------------
 * Pages shared between sequences.  The state is three device arrays of the
 * caller: page_table int32 [n_seqs][pages_per_seq], seq_len int32 [n_seqs]
 * (positions held), and refcount int32 [num_pages], the number of table
 * entries that name a page (0: free).  Entries at or beyond
 * ceil(seq_len / page_size) are not part of a sequence.
 *
 * dustin_kv_fork: sequence child[f] becomes a copy of sequence parent[f] by
 * sharing all its pages (the last, partly full one too: see dustin_kv_resize).  A fork
 * whose child is not empty (seq_len 0), is named earlier in the call, or is
 * its own parent, whose parent is a child of the call, or with an id outside
 * [0, n_seqs), is left out and raises DUSTIN_DEVFLAG_INDEX_RANGE.
 *
 * dustin_kv_resize: sequence seqs[i] gets the length new_len[i] (NULL: 0 for
 * all, the sequences are freed).
 *   - First, every sequence that shrinks gives up its pages behind the new
 *     end: refcount - 1 each, entries set to -1.
 *   - Then sequences that grow get pages, in list order, the free pages of
 *     the lowest numbers first.  A partly full last page that other entries
 *     name too is replaced by a copy of its own: copies[i] = {old page, new
 *     page} (otherwise {-1, -1}), refcount of the old page - 1; that page
 *     comes first, then the pages of the new positions.  (If all sharers of
 *     a page grow in one call, each gets a copy and the page becomes free.)
 *   - A sequence for which the free pages do not suffice, and those behind
 *     it in the list that need pages, are left as they were and raise
 *     DUSTIN_DEVFLAG_NO_PAGES.
 *   - The copied pages' rows follow for the n_layers caches in kv (all
 *     paged, with this page size and pool; page_table of the descriptors is
 *     not read).  With n_layers == 0 the caller copies.
 * An entry named before, an id or a length out of range (0 ..
 * pages_per_seq * page_size) leaves that entry out and raises
 * DUSTIN_DEVFLAG_INDEX_RANGE; a page id outside the pool is skipped and
 * raises DUSTIN_DEVFLAG_PAGE_RANGE.
 *   copies  int32 [n_list][2], device, fully overwritten
 * Limits: n_list <= 1024, num_pages <= 2^22, pages_per_seq * page_size
 * <= 2^30, n_seqs * pages_per_seq < 2^31; page_size as in dustin_kv.  Calls on one
 * state are ordered by the stream; none may overlap another. */
int dustin_kv_fork(int n_seqs, int pages_per_seq, int page_size, int num_pages,
                   int n_forks, const int32_t* parent, const int32_t* child,
                   int32_t* page_table, int32_t* seq_len, int32_t* refcount,
                   void* stream);
int dustin_kv_resize(int n_seqs, int pages_per_seq, int page_size, int num_pages,
                     int n_list, const int32_t* seqs, const int32_t* new_len,
                     int32_t* page_table, int32_t* seq_len, int32_t* refcount,
                     int32_t* copies, int n_layers, int h_kv, int d,
                     const dustin_kv* kv, void* stream);

/* ------------------------------------------------------------------------
 * A KV cache held in 4 bits: rows quantised as they are written, read back, and
 * attended to.  Not an API of the paper.
 *
 * One record per (position, kv head), dustin_kv4_record_size(d) bytes (144 for
 * d = 128, 80 for d = 64; bf16 takes 512 and 256), 16-byte aligned:
 *   d/2 bytes of codes of K (channel 2i in the low, 2i+1 in the high half of
 *   byte i), d/2 bytes of codes of V, d/16 scales of K (one per 16 channels),
 *   d/16 scales of V, zeros.
 * A value is e2m1(code) * e4m3(scale) * 2^exp, with k_exp for K and v_exp for V;
 * e2m1 has the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign (bit 3), e4m3 finite ones
 * up to 448, NaN (0x7f) and a sign that writing never sets.  All of it is exact in
 * bf16.  Scoring, page statistics, compaction and the copies of dustin_kv_resize take
 * bf16 rows only: what they are to see of such a cache is read back first, and a forked
 * page of it is copied by the caller.
 *
 * Contiguous layout (page_table == NULL): the record of (b, kv head h, position
 * j) is at data + b*stride_b + h*stride_h + j*stride_n.  Paged: position j of
 * sequence b in page p = page_table[b*pages_per_seq + j/page_size] at
 * data + p*stride_b + h*stride_h + (j % page_size)*stride_n.  Strides are in BYTES,
 * multiples of 16; k_exp and v_exp in [-64, 64].
 */
typedef struct dustin_kv4 {
  const void* data;
  int64_t stride_b;
  int64_t stride_h;
  int64_t stride_n;
  const int32_t* page_table;
  int32_t page_size;
  int32_t pages_per_seq;
  int32_t num_pages;
  int32_t k_exp;
  int32_t v_exp;
} dustin_kv4;

/* Bytes of a record; 0 for an unsupported d. */
size_t dustin_kv4_record_size(int d);

/* Writes rows into 4-bit caches: for every layer l, sequence b, kv head and
 * t < w_len[b], row t of src[l] becomes position start[b] + t of dst[l].  Of each
 * 16 channels x, with y = x * 2^-exp,
 *   scale = e4m3(min(max |y| / 6, 448)),   code = e2m1(y / scale),
 * both rounded to nearest, ties to even, beyond 6 to 6 (zeros keep their signs; a
 * scale of 0 makes all 16 zeros).  So a value is off by up to half a step of its
 * scale, |y| in (4, 6] by up to scale * 1, beyond that by what max |y| / scale
 * exceeds 6 (1/16 of the maximum; more past 2688).  16 channels that hold a NaN or
 * an infinity get the scale NaN: they read back as NaN.
 *
 *   src    host array [n_layers]: bf16 rows [b][h_kv][w][d], contiguous or paged
 *   dst    host array [n_layers]: caches of n positions
 *   start  int32 [b], device, or NULL (0 each)
 *   w_len  int32 [b], device, or NULL (w each); clamped to [0, w]
 * Positions outside [0, n) are left out (DUSTIN_DEVFLAG_INDEX_RANGE), and so are
 * pages outside the pool (DUSTIN_DEVFLAG_PAGE_RANGE).  Records are distinct: a
 * stride of 0 in dst is refused, two sequences' rows on one page are the caller's
 * to avoid.  Limits: d in {64, 128}; b * h_kv * w <= 2^30. */
int dustin_kv4_write(int n_layers, int b, int h_kv, int d, int n, int w,
                     const dustin_kv* src, const dustin_kv4* dst,
                     const int32_t* start, const int32_t* w_len, void* stream);

/* Reads rows back as bf16: for every layer l, sequence b, kv head and i < k_len[b],
 * row i of dst[l] becomes what position idx[b][i] (idx NULL: i) of src[l] stands
 * for.  Exact.  Rows from k_len[b] on are left as they were.
 *
 *   src    host array [n_layers]: caches of n positions
 *   dst    host array [n_layers]: bf16 rows [b][h_kv][k][d], contiguous or paged
 *   idx    int32 [b][k], device, or NULL; entries outside [0, n) raise
 *          DUSTIN_DEVFLAG_INDEX_RANGE, pages outside a pool
 *          DUSTIN_DEVFLAG_PAGE_RANGE, and leave their row as it was
 *   k_len  int32 [b], device, or NULL (k each); clamped to [0, k]
 * Limits: d in {64, 128}; k <= n without idx; b * h_kv * k <= 2^30. */
int dustin_kv4_read(int n_layers, int b, int h_kv, int d, int n, int k,
                    const dustin_kv4* src, const dustin_kv* dst, const int32_t* idx,
                    const int32_t* k_len, void* stream);

/* Verification attention over a 4-bit cache:
 *   o[b][h][t] = softmax over [positions idx[b][0..k_len[b]), window 0..t]
 *                of scale * q . K, times V;   lse = log sum exp (natural)
 * idx NULL takes positions 0 .. k_len[b] - 1 (the whole cache, or w = 1 rows of a
 * decoding step); the window part, where win is given, is as in the *_window calls:
 * bf16 [b][h_kv][w][d] through win->stride_b/h/n, positions 0..t only.  (A serving
 * loop keeps the window in bf16 and writes the accepted rows to the cache.)
 *
 *   q      bf16 [b][h_q][w][d], device (contiguous); o like q; lse fp32 [b][h_q][w]
 *   kv     one dustin_kv4 of n positions; ignored (may be NULL) if k is 0
 *   idx    int32 [b][k], device, or NULL; in any order.  Entries outside [0, n) are
 *          left out (DUSTIN_DEVFLAG_INDEX_RANGE), and pages outside the pool
 *          (DUSTIN_DEVFLAG_PAGE_RANGE); an entry that repeats counts each time
 *   k_len  int32 [b], device, or NULL (k each); clamped to [0, k]
 * Records behind the lengths are never used, whatever they hold.  A row that sees
 * no position, or only scores of -inf, gives o = 0, lse = -inf.  A row with a
 * score that is NaN or +inf gives NaN, o and lse (scores beyond fp32, in units of
 * log 2, count as infinite, and so do products q . K of the window).
 * DUSTIN_ATTN_KV_READY is accepted, without effect.  Sums are taken in a
 * fixed order: equal calls give equal bits.
 * Precision: cached values enter exactly, q as well (entries 2^-37 below their row's
 * largest are rounded); scores, maxima, sums and partial results are fp32.  A
 * weight of a cached position is rounded to f16 for its product with V (by 2^-11,
 * or by 2^-33 of the row's largest weight so far), and o to bf16 once.
 * Where a row's largest |q| * scale * 2^k_exp passes 2^140, its scores are those of
 * 2^140 (they may still be infinite).
 * Limits: as dustin_sparse_verify_attn; with k > 0, scale * 2^k_exp in [2^-120, 2^126]
 * (DUSTIN_ERR_SHAPE); k <= n without idx; k <= 2^27; b <= 2^20;
 * (b * h_kv * blocks of 64 query rows) * (k / 128 + 1) <= 2^30, and with k > 2^25 at
 * most 256 such blocks (an SM's share of longer ones could outlast a wait's second); a
 * workspace of 2^35 bytes.
 * Workspace: dustin_kv4_verify_attn_workspace_size (with or without win, idx);
 * its content need not be kept, and calls that may run at the same time (two
 * streams, two captured graphs) have one each. */
size_t dustin_kv4_verify_attn_workspace_size(int b, int h_q, int h_kv, int d, int w,
                                             int k);
int dustin_kv4_verify_attn(int b, int h_q, int h_kv, int d, int w, int n, int k,
                           const void* q, const dustin_kv4* kv, const int32_t* idx,
                           const int32_t* k_len, const dustin_kv* win, float scale,
                           void* o, float* lse, void* ws, size_t ws_bytes,
                           unsigned flags, void* stream);

/* ------------------------------------------------------------------------
 * Log probabilities of given tokens, with the entropy of each row and its most
 * likely tokens, from logits: what a serving loop reports beside the tokens that
 * dustin_verify_tokens accepts, and scores a prompt with.  Not an API of the paper.
 *
 * With z = scale * logits[b][t] (scale: an inverse temperature):
 *   lse[b][t]          = log sum_j exp(z_j)
 *   logprobs[b][t][i]  = z[tokens[b][t][i]] - lse
 *   entropy[b][t]      = -sum_j p_j log p_j,  p = softmax(z), 0 log 0 = 0
 *   top_ids[b][t][0..top), top_logprobs: the largest logits in descending order,
 *                        equal ones (-0 equals +0) by ascending id
 * Logits of -inf have no mass (logprob -inf); they are alternatives where the
 * others do not suffice.  A row of -inf alone has lse and all logprobs -inf and
 * entropy 0.  A row with a NaN or +inf has lse, logprobs and entropy NaN; NaN logits
 * are no alternatives (places left over: id -1, NaN).  A token outside
 * [0, vocab) has logprob -inf and raises DUSTIN_DEVFLAG_INDEX_RANGE, but -1 (no
 * token) raises nothing.
 *
 *   logits  [b][w][vocab] of `dtype` (DUSTIN_DTYPE_*), device; row (i, t) at element
 *           i*stride_b + t*stride_w, entries contiguous
 *   n_rows  int32 [b], device, or NULL (w each): rows t >= n_rows[b] are not read
 *           and their outputs left as they were
 *   tokens  int32 [b][w][m];  logprobs fp32 [b][w][m]  (may be NULL if m is 0)
 *   entropy, lse  fp32 [b][w], or NULL
 *   top_ids int32 [b][w][top];  top_logprobs fp32 [b][w][top]  (NULL if top is 0)
 * Rows may start at any element; they are read in aligned words of 16 bytes, so
 * bytes beside a row may be read too (never used).  Equal calls give equal bits.
 * Precision: weights and sums are fp32.  lse and the log probabilities are off by 4e-5
 * + 2^-22 of their size at most, the entropy by 4e-5 (1 + entropy), mostly by some 1e-7;
 * 2^-22 more for each 16384 entries (8192 in fp32) at whose end a thread's largest has
 * grown, which matters for rows of millions that rise all along.  These are absolute:
 * of a token with probability 1 - 1e-9 the log probability may be 0, and the entropy.
 * b == 0 or w == 0 is a no-op.  Limits: 1 <= vocab <= 2^30, b * w <= 2^27; m <= 512;
 * top <= min(vocab, 64); 0 < scale <= 2^100.  No workspace. */
int dustin_token_logprobs(int b, int w, int vocab, int dtype, const void* logits,
                          int64_t stride_b, int64_t stride_w, float scale,
                          const int32_t* n_rows, int m, const int32_t* tokens,
                          float* logprobs, float* entropy, float* lse, int top,
                          int32_t* top_ids, float* top_logprobs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DUSTIN_H_ */
