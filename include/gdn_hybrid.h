/*
 * gdn_hybrid.h -- C ABI of the other token mixers of a hybrid model on MI355X (gfx950): the gated
 * linear recurrence (one decay per channel and token) over prompts, with gradients and for single
 * tokens; the RMS norm of each query and key head with the rotation of its position, with gradients
 * and on the way into a paged cache; attention of one new token over such a cache.
 *
 * The rules are those of gdn_layer.h: DEVICE pointers, memory of the caller, calls that only enqueue
 * kernels on `stream` (of the current device), row views with strides in elements and 16-byte aligned
 * address and stride, contiguous arrays named [..], checks on the host before anything is enqueued.
 * Malformed cu_seqlens, slots, page tables or lengths give wrong results but no access outside the
 * caller's buffers. Results are the same bits on every run (no atomics). Rows of no sequence are left as they
 * were. A NaN stays in its channel and sequence (and its channel of dlambda), in its row and
 * head (and dwq or dwk), or in its sequence and the query heads that read it. Calls that may run at the same time need workspaces of
 * their own.
 */
#ifndef GDN_HYBRID_H
#define GDN_HYBRID_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The gated linear recurrence, per sequence and channel, with s the sigmoid:
 *
 *   L_t = rate softplus(lambda) s(r_t)          the decay's exponent
 *   a_t = exp(-L_t),  w_t = sqrt(1 - a_t^2)     the decay and the input's weight
 *   h_t = a_t h_{t-1} + w_t s(i_t) x_t,  y_t = h_t
 *
 * starting from h0 (zero when NULL). The first token of a sequence that is `fresh` enters with weight
 * one and no decay, h = s(i) x (its h0 is not read). x, r, i, y: [rows][channels] in dtype, a row
 * stride below 2^23 bytes; sums and states are float32, 1 - a and 1 - s are formed without cancellation. What strong decays
 * leave of a state (or of a gradient from behind) is off by some 2^-24 of the state in front of them, not of itself. rate
 * softplus(lambda) counts up to 2^100.
 */
typedef struct {
  int32_t N;        /* sequences (>= 0) */
  int32_t T;        /* tokens per sequence when cu_seqlens is NULL; ignored otherwise */
  int64_t T_total;  /* rows, up to 2^28 */
  const int32_t* cu_seqlens; /* DEVICE int32 [N + 1] as in gdn_problem, or NULL; empty sequences allowed */
  int32_t channels; /* a positive multiple of 8, below 2^23 bytes; (N + 1) ceil(channels / 32) + 512 up to 2^23 */
  int32_t dtype;    /* gdn_dtype of x, r, i, y and their gradients */
  float rate;       /* finite, > 0 */
  const float* lambda;   /* [channels], 16-byte aligned */
  const int32_t* fresh;  /* DEVICE int32 [N], nonzero: a fresh sequence; or NULL (none is) */
} gdn_glr_problem;

/* Bytes of device workspace (scratch, 256-byte aligned) of gdn_glr_fwd and gdn_glr_bwd, and of the
 * saved states that gdn_glr_fwd writes for gdn_glr_bwd; 0 for an invalid problem. */
size_t gdn_glr_fwd_workspace_bytes(const gdn_glr_problem* p);
size_t gdn_glr_bwd_workspace_bytes(const gdn_glr_problem* p);
size_t gdn_glr_state_bytes(const gdn_glr_problem* p);

/*
 * Forward over prompts. h0 (float32 [N][channels] or NULL) and h_T (or NULL to skip) 16-byte aligned;
 * they must not overlap. y may be the very view (address and stride) of x, r or i. states:
 * gdn_glr_state_bytes bytes, 16-byte aligned, kept unchanged for gdn_glr_bwd, or NULL when no backward
 * follows. The workspace may be NULL where its size query returns 0 (in gdn_glr_bwd too).
 */
gdn_status gdn_glr_fwd(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                       const void* i, int64_t i_rs, const float* h0, void* y, int64_t y_rs, float* h_T,
                       void* states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward: gradients for dy [rows][channels] and dh_T (float32 [N][channels], or NULL = zeros). The
 * inputs and states must be those of the forward call. Writes dx, dr, di [rows][channels] (dtype; each
 * may be the very view of an input), dlambda float32 [channels] (NULL to skip; tokens summed in a fixed
 * order, in 64 bits between the chunks' parts) and dh0 (or NULL to skip; it must not overlap dh_T).
 * A gradient of the decay's exponent is taken as zero where the exponent itself is.
 */
gdn_status gdn_glr_bwd(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                       const void* i, int64_t i_rs, const void* states, const void* dy, int64_t dy_rs,
                       const float* dh_T, void* dx, int64_t dx_rs, void* dr, int64_t dr_rs, void* di,
                       int64_t di_rs, float* dlambda, float* dh0, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * One step for each of p->N rows (p->T == 1, p->T_total == p->N, cu_seqlens NULL; fresh is per row).
 * state: float32 [n_slots][channels], 16-byte aligned, updated in place; slot_idx: int32 [N] or NULL
 * (row n -> slot n, n_slots >= N). A row whose slot is outside [0, n_slots) is skipped: its y row and
 * every state stay untouched. Two rows of one slot race (their result is undefined). y may be the very
 * view of x, r or i.
 */
gdn_status gdn_glr_decode(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                          const void* i, int64_t i_rs, float* state, int32_t n_slots, const int32_t* slot_idx,
                          void* y, int64_t y_rs, void* stream);

/*
 * The norm of each query and key head with the rotation of its position. A head v of D values becomes
 *   n = v / sqrt(mean(v^2) + eps) * w          (w: wq or wk, float32 [D]; NULL = ones)
 * and of its first `rot` values the pairs (j, j + rot / 2), or (2 j, 2 j + 1) with `adjacent`,
 *   (n_a, n_b) -> rope_scale (n_a cos - n_b sin, n_a sin + n_b cos)  at the angle position * freq[j];
 * the values behind stay. Angles and their reduction are float64.
 */
typedef struct {
  int64_t rows;       /* up to 2^25 - 2; rows (Hq + 2 Hk) < 2^31, Hq + 2 Hk < 2^21 */
  int32_t Hq, Hk, D;  /* heads and head size: a multiple of 16 up to 256 */
  int32_t rot;        /* values of a head that are rotated: a multiple of 16, 0 .. D */
  int32_t adjacent;   /* 0: pairs (j, j + rot / 2); else (2 j, 2 j + 1) */
  float eps;          /* finite, >= 0 */
  float rope_scale;   /* finite */
  int32_t dtype;      /* gdn_dtype of the row views and pages */
  const int32_t* positions; /* DEVICE int32 [rows]; may be NULL when rot is 0 */
  const double* freq;       /* DEVICE float64 [rot / 2], finite; may be NULL when rot is 0 */
  const float *wq, *wk;     /* [D], 16-byte aligned, or NULL */
} gdn_qk_rope_problem;

/* q, qo: [rows][Hq*D]; k, ko: [rows][Hk*D]. An output may be the very view of its own input (qo of q, ko
 * of k) and must not overlap an input or another output otherwise. */
gdn_status gdn_qk_rope_fwd(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                           void* qo, int64_t qo_rs, void* ko, int64_t ko_rs, void* stream);

/* Gradients dq, dk (dtype; dq may be the very view of q or dqo, dk of k or dko) and dwq, dwk (float32 [D],
 * each NULL to skip) for dqo and dko. The workspace (256-byte aligned) is needed for dwq or dwk only. */
size_t gdn_qk_rope_bwd_workspace_bytes(const gdn_qk_rope_problem* p);
gdn_status gdn_qk_rope_bwd(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                           const void* dqo, int64_t dqo_rs, const void* dko, int64_t dko_rs, void* dq, int64_t dq_rs,
                           void* dk, int64_t dk_rs, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * The serving form: queries to rows, keys (normalised and rotated) and values (as they are) into pages, and nowhere else,
 * [n_pages][Hk][page_size][D] (dtype, 16-byte aligned; k_pages and v_pages are different buffers; of the head sizes,
 * gdn_paged_attn_decode reads 32, 64, 128 and 256). v:
 * [rows][Hk*D]. where: int32 [rows], a row's place page * page_size + offset; a row whose place is outside
 * [0, n_pages * page_size), -1 for instance, is not cached (its query is written all the same). Two rows
 * of one place race. n_pages * page_size * Hk < 2^32, n_pages * page_size < 2^31.
 */
gdn_status gdn_qk_rope_cache(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                             const void* v, int64_t v_rs, void* qo, int64_t qo_rs, void* k_pages, void* v_pages,
                             int32_t n_pages, int32_t page_size, const int32_t* where, void* stream);

/*
 * Attention of one new token per sequence over a paged cache. Sequence n holds lens[n] tokens, token t in
 * page page_table[n][t / page_size] at t % page_size; query head h reads key head h / (Hq / Hk):
 *   z_t = scale q . k_t,  out = sum_t exp(z_t - lse) v_t,  lse = log sum_t exp(z_t)
 * over the last `window` of its tokens (all when window is 0). A length counts as at least 0 and at most
 * max_len; tokens of a page outside [0, n_pages) are left out. Where nothing is left, out is zero and
 * lse minus infinity. Weights and sums are float32. The cache is read once for every 16 query heads of a key head.
 */
typedef struct {
  int32_t N;           /* sequences (>= 0); N Hq < 2^24, 6 N Hk ceil(Hq / (16 Hk)) < 2^24 - 1024 */
  int32_t Hq, Hk, D;   /* Hq % Hk == 0; head size 32, 64, 128 or 256 */
  int32_t page_size;   /* tokens per page (>= 1) */
  int32_t n_pages;     /* pages of the pool (>= 0); n_pages * page_size * Hk < 2^32, n_pages * page_size < 2^31 */
  int32_t max_pages;   /* entries per row of page_table; max_pages * page_size < 2^31 */
  int32_t max_len;     /* upper bound of lens, 0 .. max_pages * page_size, up to 2^30: sizes the launch */
  int32_t window;      /* tokens seen, or 0 = all */
  float scale;         /* finite */
  int32_t dtype;       /* gdn_dtype of q, out and the pages */
  const int32_t* page_table; /* DEVICE int32 [N][max_pages] */
  const int32_t* lens;       /* DEVICE int32 [N] */
} gdn_paged_problem;

/* Bytes of workspace (scratch, 256-byte aligned; 0: none is needed). */
size_t gdn_paged_attn_workspace_bytes(const gdn_paged_problem* p);

/* q, out: [N][Hq*D]; they must not overlap. k_pages, v_pages: [n_pages][Hk][page_size][D], 16-byte aligned. lse: float32
 * [N][Hq] or NULL. */
gdn_status gdn_paged_attn_decode(const gdn_paged_problem* p, const void* q, int64_t q_rs, const void* k_pages,
                                 const void* v_pages, void* out, int64_t out_rs, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_HYBRID_H */
