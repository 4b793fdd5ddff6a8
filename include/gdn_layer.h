/*
 * gdn_layer.h -- C ABI of the operators around the recurrence of a linear-attention layer on
 * MI355X (gfx950): the selective state space scan (prompts, training, single tokens), the
 * causal conv1d + SiLU with a carried window, the gated RMS norm behind a recurrence and the
 * residual addition with the next block's RMS norm.
 *
 * The rules are those of gdn.h, with its status codes and types: every pointer is a DEVICE
 * pointer; the caller owns all memory; a call only enqueues kernels on `stream` (it never
 * allocates, frees or synchronises); rows are row-strided views whose strides are in elements,
 * 16-byte aligned in address and stride; float32 arrays named [..] are contiguous; arguments
 * are checked on the host before anything is enqueued; a malformed cu_seqlens or slot gives
 * wrong results but no access outside the caller's buffers. The scan works on chunks of 64 tokens: a
 * NaN or an infinity stays in its sequence and head (in b and c: in its group of heads), but may reach
 * the other rows of its chunk. The device that owns the stream has
 * to be current. Results are the same bits on every run (no atomics).
 */
#ifndef GDN_LAYER_H
#define GDN_LAYER_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The selective state space scan, per sequence and head h, with b and c of key head
 * kh = h / (Hv / Hk) (shared by the Hv / Hk heads of a group):
 *
 *   D_t = softplus(dt_t + dt_bias[h])           the step
 *   a_t = exp(-exp(a_log[h]) D_t)               the decay
 *   S_t = a_t S_{t-1} + b_t (x) (D_t x_t)       (Dk x Dv, stored key-major, float32)
 *   y_t = S_t^T c_t + d_skip[h] x_t
 *
 * starting from S0 (zero when NULL). x, y: [rows][Hv*Dv]; b, c: [rows][Hk*Dk]; dt: float32
 * [T_total][Hv]; a row stride is below 2^25 bytes. Sums and states are float32; products of bfloat16 inputs run on the matrix
 * cores with every float32 factor split over bfloat16 operands, three where the result is float32 (24 bits), two
 * where it is a bfloat16 row, which so carries no rounding but its own.
 */
typedef struct {
  int32_t N;        /* sequences (>= 0) */
  int32_t T;        /* tokens per sequence when cu_seqlens is NULL; ignored otherwise */
  int64_t T_total;  /* rows */
  const int32_t* cu_seqlens; /* DEVICE int32 [N + 1] as in gdn_problem, or NULL; empty sequences allowed */
  int32_t Hk, Hv;   /* groups (heads of b and c) and heads of x; Hv % Hk == 0 */
  int32_t Dk, Dv;   /* state size and head size, each one of 16, 32, 64, 128; (N + 8) Hv, twice that for
                       Dv = 128, and (T_total / 64 + N) Hv below 2^23; T_total up to 2^28 */
  int32_t dtype;    /* gdn_dtype of x, b, c, y and their gradients */
  const float* a_log;   /* [Hv] */
  const float* dt_bias; /* [Hv] or NULL (none) */
  const float* d_skip;  /* [Hv] or NULL (none) */
} gdn_ssm_problem;

/* Bytes of device workspace (scratch, 256-byte aligned) of gdn_ssm_fwd and gdn_ssm_bwd, and of
 * the saved states that gdn_ssm_fwd writes for gdn_ssm_bwd; 0 for an invalid problem. */
size_t gdn_ssm_fwd_workspace_bytes(const gdn_ssm_problem* p);
size_t gdn_ssm_bwd_workspace_bytes(const gdn_ssm_problem* p);
size_t gdn_ssm_chunk_state_bytes(const gdn_ssm_problem* p);

/*
 * Forward over prompts. Outputs must not overlap inputs or one another (here and in gdn_ssm_bwd). S0 (float32 [N][Hv][Dk][Dv] or NULL) and S_T (or NULL to skip) 16-byte
 * aligned; they must not overlap. chunk_states: gdn_ssm_chunk_state_bytes bytes, 16-byte
 * aligned, kept unchanged for gdn_ssm_bwd, or NULL when no backward follows. The workspace may
 * be NULL where its size query returns 0.
 */
gdn_status gdn_ssm_fwd(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                       const void* c, int64_t c_rs, const float* dt, const float* S0, void* y, int64_t y_rs,
                       float* S_T, void* chunk_states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward: gradients of the forward's inputs for dy [rows][Hv*Dv] and dS_T (float32, or NULL =
 * zeros). The inputs and chunk_states must be those of the forward call. Writes dx [rows][Hv*Dv],
 * db, dc [rows][Hk*Dk] (dtype; a group's heads summed in float32, rounded once), ddt float32
 * [T_total][Hv], da_log, ddt_bias, dd_skip float32 [Hv] (each NULL to skip) and dS0 (or NULL to
 * skip; it must not overlap dS_T). Sums over tokens run in a fixed order: in float32 inside a chunk, of the
 * chunks' partials (da_log, ddt_bias, dd_skip) in 64 bits.
 */
gdn_status gdn_ssm_bwd(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                       const void* c, int64_t c_rs, const float* dt, const void* chunk_states,
                       const void* dy, int64_t dy_rs, const float* dS_T, void* dx, int64_t dx_rs, void* db,
                       int64_t db_rs, void* dc, int64_t dc_rs, float* ddt, float* da_log, float* ddt_bias,
                       float* dd_skip, float* dS0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One step of the scan for each of p->N rows (p->T == 1, p->T_total == p->N, cu_seqlens NULL).
 * state: float32 [n_slots][Hv][Dk][Dv], 16-byte aligned, updated in place; slot_idx: int32 [N] or
 * NULL (row n -> slot n, n_slots >= N). A row whose slot is outside [0, n_slots) is skipped: its
 * y row and every state stay untouched. Two rows of one slot race (their result is undefined). y may be
 * x's very view and must not overlap any other argument.
 */
gdn_status gdn_ssm_decode(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                          const void* c, int64_t c_rs, const float* dt, float* state, int32_t n_slots,
                          const int32_t* slot_idx, void* y, int64_t y_rs, void* stream);

/*
 * Causal depthwise conv1d + SiLU over prompts that continue: as gdn_conv1d_silu_fwd, with a bias
 * (float32 [channels] or NULL) and with the K - 1 rows before each sequence in
 * first [N][K - 1][channels] (dtype; oldest row first; NULL = zeros). last [N][K - 1][channels]
 * (NULL to skip) receives the rows that a continuation needs: the last K - 1 rows of first and x
 * together. first and last are 16-byte aligned; y and last must not overlap one another or an input.
 * There is no backward of this form: gdn_conv1d_silu_bwd is the gradient of sequences that start empty,
 * without a bias, and SiLU's derivative depends on both.
 */
gdn_status gdn_conv1d_silu_prompt(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w,
                                  const float* bias, const void* first, void* y, int64_t y_rs, void* last,
                                  void* stream);

/*
 * The same for one token of each of p->N sequences (p->T == 1, p->T_total == p->N, cu_seqlens
 * NULL; y may be x's very view; state overlaps neither): state [n_slots][K - 1][channels] (dtype, 16-byte aligned) holds each slot's last rows,
 * oldest first, and is moved on by one row in place. Slots as in gdn_ssm_decode. For K == 1 there
 * is no window: state may be NULL (rows are skipped by n_slots all the same).
 */
gdn_status gdn_conv1d_silu_decode(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w,
                                  const float* bias, void* state, int32_t n_slots, const int32_t* slot_idx,
                                  void* y, int64_t y_rs, void* stream);

/*
 * RMS norms. A row holds `groups` groups of `width` values; each group is normalised by itself:
 * norm(v) = v / sqrt(mean(v^2) + eps) * w, with w float32 [width] for every group (shared != 0) or
 * [groups][width]. width: a multiple of 8, up to 16384; rows * groups < 2^31.
 */
typedef struct {
  int64_t rows;
  int32_t groups, width;
  int32_t shared;      /* one weight row for all groups */
  int32_t gate_first;  /* gated norm: 0: norm(x) silu(z); 1: norm(x silu(z)) */
  float eps;           /* finite, >= 0 */
  float scale;         /* residual scale of the add norm; finite */
  int32_t dtype;       /* gdn_dtype of the row views */
} gdn_norm_problem;

/* Bytes of workspace (256-byte aligned) of the two backward calls for this problem. */
size_t gdn_gated_norm_bwd_workspace_bytes(const gdn_norm_problem* p);
size_t gdn_add_norm_bwd_workspace_bytes(const gdn_norm_problem* p);

/* The norm behind a recurrence with its gate: y = norm(x) silu(z), or norm(x silu(z)). An output
 * may be the very view of an input of the same call, address and stride, and must not overlap one otherwise,
 * nor another output (here and in the calls below). */
gdn_status gdn_gated_norm_fwd(const gdn_norm_problem* p, const void* x, int64_t x_rs, const void* z, int64_t z_rs,
                              const float* w, void* y, int64_t y_rs, void* stream);
/* dx, dz (dtype) and dw (float32, w's shape; NULL to skip) for dy. */
gdn_status gdn_gated_norm_bwd(const gdn_norm_problem* p, const void* x, int64_t x_rs, const void* z, int64_t z_rs,
                              const float* w, const void* dy, int64_t dy_rs, void* dx, int64_t dx_rs, void* dz,
                              int64_t dz_rs, float* dw, void* workspace, size_t workspace_bytes, void* stream);

/* The residual addition and the norm before the next block (groups == 1):
 *   res = h + scale s y  (s: float32 [width] or NULL = ones), rounded to dtype as stored,
 *   out = norm(res)      (of the stored values). */
gdn_status gdn_add_norm_fwd(const gdn_norm_problem* p, const void* h, int64_t h_rs, const void* y, int64_t y_rs,
                            const float* s, const float* w, void* res, int64_t res_rs, void* out, int64_t out_rs,
                            void* stream);
/* From dout (gradient of out) and dres (gradient of res from the residual path; NULL = zeros):
 *   dh = norm'(dout) + dres,  dy = scale s dh (NULL to skip),  dw [width] (NULL to skip),
 *   ds[c] = scale sum_rows dh y  [width] (NULL to skip; y is read only for it and may be NULL otherwise). */
gdn_status gdn_add_norm_bwd(const gdn_norm_problem* p, const void* res, int64_t res_rs, const void* y, int64_t y_rs,
                            const float* s, const float* w, const void* dout, int64_t dout_rs, const void* dres,
                            int64_t dres_rs, void* dh, int64_t dh_rs, void* dy, int64_t dy_rs, float* dw, float* ds,
                            void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H */
