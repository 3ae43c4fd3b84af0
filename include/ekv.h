/*
 * ekv.h — C ABI of the EntmaxKV support-aware paged α-entmax decode library
 * (libekv.so, hand-written CUDA for sm_100a).
 *
 * Source of the method: "Résumé Technique : EntmaxKV – Décodage Conscient du
 * Support pour l'Attention Entmax" (gist.science/fr/paper/2605.21649), cited
 * below as [EntmaxKV] with the section that defines each operation.  The page
 * states the problem (a paged KV cache, a decode query, per-page metadata, a
 * top-k budget k or a margin Δ, α) and prints no formula and no API; the
 * formulas used are stated beside each call.
 *
 * Conventions shared by every call
 * --------------------------------
 * Ownership   The caller owns every buffer.  All pointers named "device" point
 *             to CUDA device memory; the library never allocates and keeps no
 *             state between calls except the sticky device error word read by
 *             ekv_get_error().
 * Streams     `stream` is a cudaStream_t passed as void* (NULL = legacy
 *             default stream).  Every call only enqueues work on it and never
 *             synchronises, except ekv_get_error().
 * Errors      Host-side validation runs before any launch and returns
 *             EKV_ERR_INVALID_ARG / EKV_ERR_UNSUPPORTED / EKV_ERR_WORKSPACE
 *             without touching the device.  A failed launch returns
 *             EKV_ERR_CUDA.  Data-dependent faults found on the device (a page
 *             id outside the pool, a sequence length outside 1..max_pages·S, a
 *             Gaussian selection larger than `cap`) never trap: the kernel skips
 *             the access, clamps, and ORs a bit into the device error word.
 * Dtypes      EKV_BF16 or EKV_F32 for the K/V pools, the metadata pools and
 *             the query.  Scores, bounds, thresholds and outputs are fp32.
 * Indices     Pages named in `sel` are *logical* page indices of the
 *             sequence; page_table maps them to physical pages.
 * Units       A unit is one (sequence b, KV head h) pair, u = b·Hkv + h.
 *             Query head hq belongs to KV head hq / G with G = Hq / Hkv.
 *
 * Memory layouts (row-major, dense)
 * ---------------------------------
 *   k_pool, v_pool [num_phys_pages, Hkv, S, d]
 *   box            [Hkv, num_phys_pages, 2, d]   row 0 = k_max, row 1 = k_min
 *   mom            [Hkv, num_phys_pages, 2, d]   row 0 = mean,  row 1 = variance
 *                  (head-major: one head's rows of consecutive physical pages
 *                  are adjacent, so scoring a sequence reads them in order)
 *   page_table     [batch, max_pages] int32, seq_lens [batch] int32
 *   q              [batch, Hq, d]
 *   ub             [batch, Hkv, max_pages] fp32
 *   sel            [batch, Hkv, cap] int32 (ascending), n_sel [batch, Hkv]
 *   out            [batch, Hq, d] fp32
 */
#ifndef EKV_H
#define EKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define EKV_API __attribute__((visibility("default")))

typedef enum {
  EKV_OK = 0,
  EKV_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, α ≤ 1, k < 1, ... */
  EKV_ERR_UNSUPPORTED = 2, /* d ∉ {64,128}, S ∉ {16,32}, G ∉ {1,2,4,8,16}, β not integer */
  EKV_ERR_WORKSPACE = 3,   /* ws too small or not 256-byte aligned */
  EKV_ERR_CUDA = 4,        /* a kernel launch or CUDA runtime call failed */
  EKV_ERR_TIMEOUT = 5      /* reserved: a bounded device wait gave up */
} ekv_status;

typedef enum { EKV_F32 = 0, EKV_BF16 = 1 } ekv_dtype;

/* Bits of the sticky device error word (ekv_get_error). */
#define EKV_EFLAG_BAD_PAGE 1u      /* page_table entry outside [0, num_phys_pages) */
#define EKV_EFLAG_BAD_LEN 2u       /* seq_lens entry outside [1, max_pages·S] */
#define EKV_EFLAG_SEL_OVERFLOW 4u  /* Gaussian policy kept more than cap pages */
#define EKV_EFLAG_BAD_SEL 8u       /* sel entry outside [0, pages of the sequence) */
#define EKV_EFLAG_TIMEOUT 16u      /* a bounded wait on an asynchronous copy gave up */
#define EKV_EFLAG_BAD_POS 32u      /* a token's position has no row in the rotation table */

/* The paged KV cache and its per-page metadata pools (all device memory). */
typedef struct {
  int32_t dtype;          /* ekv_dtype of k_pool, v_pool, box, mom and q */
  int32_t head_dim;       /* d ∈ {64, 128} */
  int32_t page_size;      /* S ∈ {16, 32} tokens per page */
  int32_t num_kv_heads;   /* Hkv ≥ 1 */
  int32_t num_phys_pages; /* pages in each pool */
  void* k_pool;
  void* v_pool;
  void* box;
  void* mom;
} ekv_cache;

/* The batch of sequences: page tables and lengths (device memory). */
typedef struct {
  const int32_t* page_table; /* [batch, max_pages] physical page of each logical page */
  const int32_t* seq_lens;   /* [batch] tokens, including the one being decoded */
  int32_t batch;
  int32_t max_pages;
} ekv_seqs;

/*
 * ekv_build_page_meta — [EntmaxKV] §2.A, "Bornes de Boîte Englobante" and
 * "Statistiques Gaussiennes".  For every page p < ⌈L_b/S⌉ of every sequence
 * and every KV head, over the n_p = min(S, L_b − p·S) valid tokens, writes
 *   box: k_max_j, k_min_j (exact);
 *   mom: μ_j = (1/n_p)Σ_t k_tj and the population variance
 *        σ²_j = (1/n_p)Σ_t (k_tj − μ_j)²,
 * both accumulated in float64 in token order and rounded once (nearest-even)
 * to the cache dtype.  Used after prefill; reads all of K.
 */
EKV_API ekv_status ekv_build_page_meta(const ekv_cache* cache, const ekv_seqs* seqs, void* stream);

/*
 * ekv_append — the cache append of a decode step, fused with the metadata
 * update of [EntmaxKV] §2.A.  k_new, v_new: device [batch, Hkv, d] in the cache
 * dtype.  Writes token L_b − 1 of every sequence (seq_lens already counts it)
 * into its page, then recomputes box/mom of that page over its valid tokens
 * exactly as ekv_build_page_meta does.
 */
EKV_API ekv_status ekv_append(const ekv_cache* cache, const ekv_seqs* seqs, const void* k_new,
                              const void* v_new, void* stream);

/*
 * ekv_score_pages — [EntmaxKV] §2.A, the bounding-box upper bound.  For query
 * head h and page p: ub_{p,h} = scale·Σ_j max(q_hj·kmin_pj, q_hj·kmax_pj),
 * an upper bound of every token score scale·q_h·k of the page.  The page
 * score of a KV head is the max over the G query heads of its group:
 * ub[b, kvh, p] for p < ⌈L_b/S⌉ (entries past that are not written).
 * q: device [batch, Hq, d]; ub: device fp32 [batch, Hkv, max_pages].
 */
EKV_API ekv_status ekv_score_pages(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                   int32_t num_q_heads, float scale, float* ub, void* stream);

/*
 * ekv_select_topk — [EntmaxKV] §2.B.1, "Sélection de Pages Top-k": per unit,
 * the k pages with the largest ub (ties to the lower logical index; all pages
 * when ⌈L_b/S⌉ ≤ k), written ascending to sel[b, kvh, 0..n_sel) with
 * n_sel = min(k, ⌈L_b/S⌉).  page_size S turns seq_lens into page counts.
 * ub: device [batch, Hkv, max_pages] (ekv_score_pages); sel: device
 * [batch, Hkv, k]; n_sel: [batch, Hkv].  ws: ekv_workspace_bytes(
 * EKV_OP_SELECT_TOPK, ..., cap = k) bytes, which is 0 (ws may be NULL) up to
 * 16384 pages per sequence; longer sequences with that scratch are selected
 * in two stages (chunks of 8192 pages keep their k best, then k among those),
 * without it in one slower stage.
 */
EKV_API ekv_status ekv_select_topk(const ekv_seqs* seqs, int32_t num_kv_heads, int32_t page_size,
                                   const float* ub, int32_t k, int32_t* sel, int32_t* n_sel,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * ekv_select_gauss — [EntmaxKV] §2.A "Statistiques Gaussiennes" + §2.B.2,
 * "Sélection Entmax Consciente de Gaussienne".  Per query head h: token scores
 * of page p are modelled as N(m, s²) with m = scale·q_h·μ_p and
 * s² = scale²·Σ_j q_hj² σ²_pj.  τ̂_h solves Σ_p n_p·E[(u − τ̂)_+^β] = 1 with
 * u ~ N((α−1)m, (α−1)²s²), β = 1/(α−1) ∈ {1,2,3,4} (else EKV_ERR_UNSUPPORTED).
 * Page p is kept when (α−1)·(m + s·√(2 ln n_p)) > τ̂_h − Δ for any head of the
 * group; if none is, the single page with the largest margin.  sel (ascending)
 * holds at most cap pages: a larger selection keeps its first cap pages and
 * sets EKV_EFLAG_SEL_OVERFLOW.  tau_hat: device fp32 [batch, Hq] (nullable).
 * ws: device scratch of ekv_workspace_bytes(EKV_OP_SELECT_GAUSS, ...) bytes.
 */
EKV_API ekv_status ekv_select_gauss(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                    int32_t num_q_heads, float scale, float alpha, float delta,
                                    int32_t cap, int32_t* sel, int32_t* n_sel, float* tau_hat,
                                    void* ws, size_t ws_bytes, void* stream);

/*
 * ekv_entmax_decode — [EntmaxKV] §2.C, "Attention Entmax Parcimonieuse".  Over
 * the valid tokens T of the selected pages (sel == NULL: every page of the
 * sequence, the full-cache decode), for every query head of the unit:
 *   z_i = scale·q·k_i,  u_i = (α−1)·z_i,
 *   τ solves Σ_{i∈T} [u_i − τ]_+^{1/(α−1)} = 1,  p_i = [u_i − τ]_+^{1/(α−1)},
 *   out = Σ_i p_i·v_i,
 * reading V only for pages that hold a token with p_i > 0 for some head of
 * the group (dense_v ≠ 0 reads every selected V page instead).
 * sel: device [batch, Hkv, cap] with n_sel entries per unit (ascending), or
 * NULL with n_sel NULL; cap bounds n_sel (max_pages when sel is NULL).
 * Outputs (device): out fp32 [batch, Hq, d]; nullable tau [batch, Hq],
 * support_count [batch, Hq] int32, support_bits uint32
 * [batch, Hq, ⌈cap·S/32⌉] (bit i of a row: token i of the selected-token list,
 * page-major, is in the support).
 * ws: ekv_workspace_bytes(EKV_OP_ENTMAX_DECODE, ...) bytes.
 */
EKV_API ekv_status ekv_entmax_decode(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                     int32_t num_q_heads, float scale, float alpha,
                                     const int32_t* sel, const int32_t* n_sel, int32_t cap,
                                     int32_t dense_v, float* out, float* tau,
                                     int32_t* support_count, uint32_t* support_bits, void* ws,
                                     size_t ws_bytes, void* stream);

/*
 * ekv_softmax_decode — softmax attention decode over the paged cache: the
 * full-cache baseline of [EKV] §4 (reading the whole cache is what sparse
 * decoding avoids), split over pages.  (ekv_softmax_decode_mod with a NULL mod
 * computes the same of a bf16 cache in two thirds of the time.)  For every query head h, o_h = Σ_i e^{z_i − m}·v_i / Σ_i e^{z_i − m}
 * with z_i = scale·q_h·k_i over every valid token of the selected pages
 * (sel = NULL with n_sel NULL: every page of the sequence; cap ≥ max_pages).
 * sel: device [batch, Hkv, cap] logical page indices with n_sel entries per
 * unit (as ekv_entmax_decode).  Outputs (device): out fp32 [batch, Hq, d];
 * lse (nullable) fp32 [batch, Hq] = m + ln Σ_i e^{z_i − m} (−inf for a
 * sequence without tokens, whose output row is 0).  bf16 caches with a page
 * size that is a multiple of 16; any other returns EKV_ERR_UNSUPPORTED.
 * ws: ekv_workspace_bytes(EKV_OP_SOFTMAX_DECODE, ...) bytes; the call clears
 * the part it needs.
 */
EKV_API ekv_status ekv_softmax_decode(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                      int32_t num_q_heads, float scale, const int32_t* sel,
                                      const int32_t* n_sel, int32_t cap, float* out, float* lse,
                                      void* ws, size_t ws_bytes, void* stream);

/*
 * Rotary position embedding.  Pairs (x1, x2) of the first rot_dim coordinates
 * of a head become (x1·c − x2·s, x2·c + x1·s) with the cosine c and sine s of
 * the token's position; the other coordinates pass unchanged.  The pairs are
 * (j, j + rot_dim/2), or (2j, 2j + 1) when interleaved ≠ 0.  The angles are
 * the caller's: row p of the table holds the rot_dim/2 cosines of position p,
 * then its rot_dim/2 sines (any frequency scaling is in the table).
 */
typedef struct {
  const float* cos_sin; /* device fp32 [max_pos, rot_dim], 16-byte aligned */
  int32_t max_pos;      /* rows; a token at a position ≥ max_pos is rotated by the
                           last row and raises EKV_EFLAG_BAD_POS */
  int32_t rot_dim;      /* a multiple of 16, 16 ≤ rot_dim ≤ d */
  int32_t interleaved;
} ekv_rope;

/*
 * New tokens of a batch, one row per token.  Rows indptr[b] .. indptr[b+1]−1
 * are the last n_b = indptr[b+1] − indptr[b] tokens of sequence b, at positions
 * L_b − n_b .. L_b − 1 (seq_lens already counts them; n_b = 0 leaves the
 * sequence alone).  Rows at and past indptr[batch] are neither read nor
 * written.  A row holds its heads densely ([Hkv, d] or [Hq, d]); the rows may
 * be strided, so the three can be views of one fused projection.
 */
typedef struct {
  const void* q;         /* device, cache dtype; NULL: no queries to rotate */
  const void* k;
  const void* v;
  void* q_out;           /* device [num_tokens, Hq, d] dense; may be q itself */
  int64_t q_stride;      /* elements from one token's row to the next */
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* indptr; /* device [batch + 1], nondecreasing; NULL: row b is the last token
                            of sequence b (unused where L_b = 0, an idle slot) */
  int32_t num_tokens;    /* rows of q, k, v and q_out */
  int32_t num_q_heads;   /* Hq (ignored when q is NULL) */
  int32_t dtype;         /* ekv_dtype of q, k, v and q_out */
} ekv_new_tokens;

/*
 * ekv_rope_append — the cache append of a decode step, a prompt or a chunk of
 * one, with the rotation applied on the way.  Rotates k (rope NULL: no
 * rotation) and writes it and v to the tokens' places in the pages; rotates q
 * into q_out; recomputes box/mom of every page that received a token over its
 * valid tokens, exactly as ekv_build_page_meta does (of the keys as stored;
 * [EntmaxKV] §2.A).  box and mom may both be NULL: no metadata is kept then.
 * The rotation runs in fp32 and is rounded once to the cache dtype.  dtype
 * must be the cache's.  Row pointers are 16-byte aligned and strides a
 * multiple of 16 bytes (else EKV_ERR_INVALID_ARG).  A sequence whose indptr
 * entries or length are inconsistent (n_b > L_b, L_b > max_pages·S, rows past
 * num_tokens) is skipped and raises EKV_EFLAG_BAD_LEN; L_b = 0 with n_b = 0 is
 * an idle slot and raises nothing.
 */
EKV_API ekv_status ekv_rope_append(const ekv_cache* cache, const ekv_seqs* seqs, const ekv_rope* rope,
                                   const ekv_new_tokens* tokens, void* stream);

/*
 * A paged cache held in 4 bits.  pool: [num_phys_pages, Hkv, S/16, R] bytes,
 * one record of R = 16·d + 128 bytes per 16 tokens: the K codes [16, d/2]
 * (coordinate 2i in the low half of byte i), the V codes [16, d/2], 16 pairs
 * (step, zero) in bf16 for K, 16 for V.  A row x of d numbers has
 *   zero = bf16(min x), step = bf16((max x − min x)/15) (0 below 1e-30),
 *   n_j = clamp(round((x_j − zero)/step), 0, 15)   (halves to the even code),
 * and stands for zero + step·n_j.  bf16() takes the numbers in 64 bits and rounds
 * them to fp32, and from there to bf16, so one within 2^-24 of the middle of two
 * bf16 numbers counts as on it.  A row with a NaN or an infinity stands for NaN
 * throughout (its codes are 0, its step is not finite); in metadata, as in
 * ekv_cache's, the extremes pass over NaN and the moments do not.  box and mom as
 * in ekv_cache, always bf16, over the values the codes stand for; k_max is
 * rounded up and k_min down, so the bounding-box bound stays a bound.  To score pages, pass an ekv_cache of
 * dtype EKV_BF16 with the same sizes, box and mom to ekv_score_pages or
 * ekv_select_gauss (they read no K).
 */
typedef struct {
  int32_t head_dim;       /* d ∈ {64, 128} */
  int32_t page_size;      /* S ∈ {16, 32} */
  int32_t num_kv_heads;
  int32_t num_phys_pages;
  void* pool;             /* device, 16-byte aligned */
  void* box;              /* device, nullable together with mom */
  void* mom;
} ekv_cache_q4;

/*
 * ekv_rope_append_q4 — ekv_rope_append into a 4-bit cache.  tokens->dtype is
 * EKV_BF16 or EKV_F32 (q_out has it too).  The codes are those of the exact
 * rotated row: borders between two codes are decided in 64 bits.
 */
EKV_API ekv_status ekv_rope_append_q4(const ekv_cache_q4* cache, const ekv_seqs* seqs, const ekv_rope* rope,
                                      const ekv_new_tokens* tokens, void* stream);

/*
 * ekv_q4_read — reads tokens of a 4-bit cache back as values: row
 * indptr[b] + i of k_out / v_out (device [num_tokens, Hkv, d] dense, out_dtype,
 * 16-byte aligned, either may be NULL) is token L_b − n_b + i of sequence b,
 * zero + step·n rounded to fp32 (and from there to bf16).  indptr (device
 * [batch + 1], not NULL) and its checks are those of ekv_new_tokens; rows it
 * does not name are left as they were.
 */
EKV_API ekv_status ekv_q4_read(const ekv_cache_q4* cache, const ekv_seqs* seqs, const int32_t* indptr,
                               int32_t num_tokens, int32_t out_dtype, void* k_out, void* v_out, void* stream);

/*
 * How scores are capped, biased and masked.  For the query token at position
 * i and the token at position j, with z = scale·q·k_j:
 *   s = softcap·tanh(z / softcap) (softcap > 0; s = z for softcap = 0)
 *       − slopes[hq]·|i − j|       (slopes not NULL),
 * and j is visible when j ≥ starts[b] and (j < prefix_lens[b] or (j ≤ i and
 * (window = 0 or i − j < window))).  NULL starts / prefix_lens count as 0.
 * Positions are those of the sequence, from 0; starts[b] is the first token
 * of the query's own document.
 */
typedef struct {
  float softcap;
  int32_t window;
  const float* slopes;        /* device fp32 [Hq], finite, nullable */
  const int32_t* prefix_lens; /* device [batch], nullable */
  const int32_t* starts;      /* device [batch], nullable */
} ekv_score_mod;

/*
 * ekv_softmax_decode_mod — ekv_softmax_decode with capped, biased and masked
 * scores, for num_q_tokens query tokens per sequence: the last T tokens of it,
 * query t at position i = L_b − T + t (a draft's tokens checked at once).
 * q: device [batch, T, Hq, d] in the cache dtype, 16-byte aligned; out: fp32
 * [batch, T, Hq, d], 16-byte aligned; lse (nullable): fp32 [batch, T, Hq].
 * mod may be NULL (causal, nothing else).  sel / n_sel / cap as
 * ekv_softmax_decode; a page named twice counts twice.  Only pages with a
 * visible token are read.  A row without a visible token (also L_b = 0, an
 * idle slot, and i < 0), or with scores of −inf alone, gives out 0 and lse −inf.
 * K and V of tokens that a row does not see never reach it, NaN and infinities
 * included.  Sums of p·v are held in fp32 with p up to 2^8, so a bf16 cache's
 * |v| times the visible tokens stays below 2^119.  bf16 caches, G·T ≤ 64,
 * max_pages·S·Hkv < 2³⁰ (cap·S < 2³⁰ with sel); anything else returns
 * EKV_ERR_UNSUPPORTED.  ws:
 * ekv_softmax_mod_workspace_bytes() bytes, 256-byte aligned, for one call at a
 * time; nothing in it outlives the call.
 */
EKV_API ekv_status ekv_softmax_decode_mod(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                          int32_t num_q_heads, int32_t num_q_tokens, float scale,
                                          const ekv_score_mod* mod, const int32_t* sel, const int32_t* n_sel,
                                          int32_t cap, float* out, float* lse, void* ws, size_t ws_bytes,
                                          void* stream);

/*
 * ekv_softmax_decode_q4 — ekv_softmax_decode_mod over a 4-bit cache: K and V
 * are the values the codes stand for (not rounded further).  q is bf16.  Steps
 * are at least 0, and V's below 2^63 (a row that sees a larger one gets NaN or
 * infinities).  scale·q, over softcap where there is one of at least 1e-30, is
 * taken up to 2^110 in size.
 */
EKV_API ekv_status ekv_softmax_decode_q4(const ekv_cache_q4* cache, const ekv_seqs* seqs, const void* q,
                                         int32_t num_q_heads, int32_t num_q_tokens, float scale,
                                         const ekv_score_mod* mod, const int32_t* sel, const int32_t* n_sel,
                                         int32_t cap, float* out, float* lse, void* ws, size_t ws_bytes,
                                         void* stream);

/*
 * Device scratch of ekv_softmax_decode_mod and ekv_softmax_decode_q4 (both
 * alike; it depends on no batch size or length).  0 when the sizes are
 * invalid or unsupported.
 */
EKV_API size_t ekv_softmax_mod_workspace_bytes(int32_t head_dim, int32_t num_kv_heads, int32_t num_q_heads,
                                               int32_t num_q_tokens);

/*
 * ekv_exactness_certificate — [EKV] §3 "Récupération du Support": the sparse
 * output equals the full-cache output when the selection holds the α-entmax
 * support.  certified[b, hq] = 1 when (α−1)·max_{p ∉ sel} ub[b, kvh, p] ≤
 * tau[b, hq] over the valid unselected pages p of unit (b, kvh = hq / G), or
 * when no valid page is left unselected; else 0.  A head whose τ is +inf (no
 * finite score among the selected tokens) is certified only in the latter
 * case.  ub: device [batch, Hkv, max_pages] unit scores from ekv_score_pages;
 * sel / n_sel / cap as for ekv_entmax_decode (non-NULL); tau: device
 * [batch, Hq] from the decode of that selection; certified: device int32
 * [batch, Hq].  max_pages above 393216 returns EKV_ERR_UNSUPPORTED.
 */
EKV_API ekv_status ekv_exactness_certificate(const ekv_seqs* seqs, int32_t num_kv_heads,
                                             int32_t page_size, int32_t num_q_heads, float alpha,
                                             const float* ub, const int32_t* sel,
                                             const int32_t* n_sel, int32_t cap, const float* tau,
                                             int32_t* certified, void* stream);

/*
 * ekv_decode_adaptive — the top-k decode with a budget that grows until the
 * output is provably the full-cache one ([EKV] §3 "Récupération du Support",
 * through ekv_exactness_certificate): page scores once, then for
 * k = k0, 2·k0, 4·k0, … (at most max_pages) the top-k selection, the sparse
 * decode and the certificate of every query head; the first k at which every
 * head of every unit is certified (or every page is selected) ends it.  The
 * count of uncertified heads is kept on the device and read back once per
 * round, so the call synchronises `stream` once per round.  Outputs are those
 * of the last round: sel device [batch, Hkv, k] (row stride k = *k_used; the
 * buffer must hold batch·Hkv·max_pages entries), n_sel [batch, Hkv], out
 * fp32 [batch, Hq, d], tau fp32 [batch, Hq], certified int32 [batch, Hq]
 * (all 1: a selection of every page is certified too); k_used: host int.  scale and
 * alpha as ekv_entmax_decode.  ws: ekv_workspace_bytes(
 * EKV_OP_DECODE_ADAPTIVE, ...) bytes (cap ignored).
 */
EKV_API ekv_status ekv_decode_adaptive(const ekv_cache* cache, const ekv_seqs* seqs, const void* q,
                                       int32_t num_q_heads, float scale, float alpha, int32_t k0,
                                       int32_t* sel, int32_t* n_sel, float* out, float* tau,
                                       int32_t* certified, int32_t* k_used, void* ws, size_t ws_bytes,
                                       void* stream);

/* Bytes of the library-owned scratch array of ekv_entmax_decode_static_ws. */
#define EKV_STATIC_WS_BYTES (16u << 20)

/*
 * ekv_entmax_decode_static_ws — ekv_entmax_decode without a caller workspace.
 * The source page has no counterpart to this call: it exists for callers
 * that cannot allocate device memory, such as a plugin inside a framework
 * that owns the device memory pool and offers no scratch buffer, or a serving
 * loop that must not call cudaMalloc once running.  Arguments and outputs are
 * those of ekv_entmax_decode; the scratch comes from one static device array
 * of EKV_STATIC_WS_BYTES bytes that every GPU loading the library holds until
 * the process exits.  A configuration whose scratch
 * (ekv_workspace_bytes(EKV_OP_ENTMAX_DECODE, ...)) exceeds that size returns
 * EKV_ERR_WORKSPACE before any device work (the limit is checked against
 * the scratch of every decode path, although the one-cluster-per-unit path,
 * taken for few units, keeps its scratch in shared memory and reads none of
 * the array; the many-unit and fp32 paths keep their scores, maxima, page
 * ids and split counters there).  All calls on a device share the array:
 * calls that overlap on the GPU race, so serialise them.  The array keeps
 * the previous call's contents; the only part that must start at zero (the
 * split counters) is reset by the call itself.  The call looks up the
 * array's device address with the device current: on the first call on a
 * device, and again on every call made outside a stream capture (so a
 * cudaDeviceReset, after which the address may change, is followed); a call
 * inside a capture uses the address found before, so make one call on each
 * device before capturing.  Allocates nothing.
 */
EKV_API ekv_status ekv_entmax_decode_static_ws(const ekv_cache* cache, const ekv_seqs* seqs,
                                               const void* q, int32_t num_q_heads, float scale,
                                               float alpha, const int32_t* sel,
                                               const int32_t* n_sel, int32_t cap, int32_t dense_v,
                                               float* out, float* tau, int32_t* support_count,
                                               uint32_t* support_bits, void* stream);

/* Selection policies of a whole decode step. */
typedef enum { EKV_POLICY_TOPK = 0, EKV_POLICY_GAUSS = 1, EKV_POLICY_FULL = 2 } ekv_policy;

typedef struct {
  int32_t policy;  /* ekv_policy */
  int32_t k;       /* top-k budget (EKV_POLICY_TOPK) */
  float delta;     /* margin Δ (EKV_POLICY_GAUSS) */
  int32_t cap;     /* pages a unit may select: k for top-k, ≤ max_pages otherwise */
  float alpha;     /* α > 1 */
  float scale;     /* score scale, usually 1/√d */
  int32_t dense_v; /* 1: read V of every selected page */
  int32_t append;  /* 1: run ekv_append(k_new, v_new) first */
} ekv_step_params;

/*
 * ekv_decode_step — one whole decode step of [EntmaxKV] §2 in stream order:
 * append (if params->append) → page scores + top-k, or the Gaussian policy,
 * or every page → sparse α-entmax attention.  sel / n_sel receive the
 * selection (device [batch, Hkv, cap] / [batch, Hkv]); out [batch, Hq, d].
 * tau (nullable) receives [batch, Hq] thresholds.  ws: ekv_workspace_bytes(
 * EKV_OP_DECODE_STEP, ...) bytes.
 */
EKV_API ekv_status ekv_decode_step(const ekv_cache* cache, const ekv_seqs* seqs,
                                   const ekv_step_params* params, const void* q,
                                   int32_t num_q_heads, const void* k_new, const void* v_new,
                                   int32_t* sel, int32_t* n_sel, float* out, float* tau, void* ws,
                                   size_t ws_bytes, void* stream);

typedef enum {
  EKV_OP_SELECT_GAUSS = 1,
  EKV_OP_ENTMAX_DECODE = 2,
  EKV_OP_DECODE_STEP = 3,
  EKV_OP_SOFTMAX_DECODE = 4,
  EKV_OP_SELECT_TOPK = 5,
  EKV_OP_DECODE_ADAPTIVE = 6
} ekv_op;

/*
 * ekv_workspace_bytes — device scratch an op needs, from the host-side sizes
 * only (cache dims, batch, max_pages, Hq, cap; for EKV_OP_DECODE_STEP `cap` is
 * params->cap).  Returns 0 when the sizes are invalid.
 */
EKV_API size_t ekv_workspace_bytes(int32_t op, const ekv_cache* cache, const ekv_seqs* seqs,
                                   int32_t num_q_heads, int32_t cap);

/*
 * ekv_step_kernel_count — how many kernels one ekv_decode_step call with these
 * arguments enqueues: the append (if params->append), the selection (2 for
 * top-k, 3 when it runs in two stages (more than 16384 pages per sequence),
 * 3 for the Gaussian policy, 0 for every page) and the decode (1 when
 * a bf16 selection fits the one-cluster-per-unit kernel, else 3).  Host-side
 * only; returns 0 when the sizes are invalid.
 */
EKV_API int32_t ekv_step_kernel_count(const ekv_cache* cache, const ekv_seqs* seqs,
                                      const ekv_step_params* params, int32_t num_q_heads);

/*
 * ekv_selftest_wait_timeout — exercises the failure path every bounded wait
 * of the library shares: one GPU thread waits, for `polls` polls (1 to
 * 1048576), on an mbarrier that nothing ever completes; the wait gives up,
 * ORs EKV_EFLAG_TIMEOUT into the device error word and the kernel returns, so
 * the context stays usable.  No source-page counterpart: a diagnostic for
 * failure detection.
 */
EKV_API ekv_status ekv_selftest_wait_timeout(uint32_t polls, void* stream);

/* Reads the sticky device error word into *flags (EKV_EFLAG_* bits) and clears
 * it.  Synchronises the device. */
EKV_API ekv_status ekv_get_error(uint32_t* flags);

/* Static description of a status code. */
EKV_API const char* ekv_status_string(ekv_status status);

#ifdef __cplusplus
}
#endif
#endif /* EKV_H */
