// layer_internal.h -- descriptors shared by the host entry points of gdn_layer.h and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Column sums of up to three planes [R][W] of float32 partials in a fixed order (norm.hip):
// o.p[plane][c] = sum_r in[plane][r][c]; a null output is skipped.
struct ColsumOut {
  float* p[3];
};
hipError_t launch_colsum(const float* in, int64_t R, int W, const ColsumOut& o, int planes, hipStream_t s);

// conv_carry.hip
struct ConvCarryArgs {
  int N, T, ch, K;  // sequences (or rows of a decode step), rows per sequence when cu is null
  int64_t rows;
  const int* cu;
  const float *w, *bias;
  const void* x;
  void* y;
  int64_t x_rs, y_rs;
  const void* first;  // [N][K - 1][ch] or nullptr
  void* last;         // [N][K - 1][ch] or nullptr
  void* state;        // decode: [n_slots][K - 1][ch]
  int n_slots;
  const int* idx;
};
hipError_t launch_conv_prompt(const ConvCarryArgs& a, int dtype, hipStream_t s);
hipError_t launch_conv_decode(const ConvCarryArgs& a, int dtype, hipStream_t s);

// norm.hip
struct NormArgs {
  int64_t rows;
  int groups, width;
  int shared, gate_first;
  float eps, scale;
  const void *x, *z;  // gated norm: x and z; add norm: h (forward) or res (backward), and y
  int64_t x_rs, z_rs;
  const float *w, *s;
  const void *g, *g2;  // upstream: dy; or dout and dres (nullptr = zeros)
  int64_t g_rs, g2_rs;
  void *o, *o2;  // y; or dx and dz; or res and out; or dh and dy (o2 nullptr = skip)
  int64_t o_rs, o2_rs;
  float *dw, *ds;  // nullptr = skip
  float* ws;
};
enum NormKind { GATE_FWD, GATE_BWD, ADD_FWD, ADD_BWD };
size_t norm_ws_bytes(const NormArgs& a, bool add);
hipError_t launch_norm(NormKind kind, const NormArgs& a, int dtype, hipStream_t s);

// ssm_decode.hip
struct SsmDecArgs {
  int N, Hv, r, Dk, Dv, n_slots;
  const void *x, *b, *c;
  int64_t x_rs, b_rs, c_rs, y_rs;
  const float *dt, *a_log, *dt_bias, *d_skip;
  float* state;
  const int* idx;
  void* y;
};
hipError_t launch_ssm_decode(const SsmDecArgs& a, int dtype, hipStream_t s);

// ssm_sweep.hip, ssm_grad.hip: everything of one forward or backward call.
struct SsmArgs {
  int N, Hk, Hv, r, Dk, Dv, T;
  int64_t T_total;
  const int* cu;
  const void *x, *b, *c, *dy;
  int64_t x_rs, b_rs, c_rs, dy_rs;
  const float *dt, *a_log, *dt_bias, *d_skip;
  const float *S0, *dST;
  void *y, *dx, *db, *dc;
  int64_t y_rs, dx_rs, db_rs, dc_rs;
  float *ST, *dS0, *ddt, *da_log, *ddt_bias, *dd_skip;
  float* sv;    // states at the chunks' starts [slot][Hv][Dk][Dv], or nullptr
  float* ws;    // workspace
};
size_t ssm_fwd_ws_bytes(const SsmArgs& a);
size_t ssm_bwd_ws_bytes(const SsmArgs& a);
size_t ssm_saved_bytes(const SsmArgs& a);
hipError_t launch_ssm_forward(const SsmArgs& a, int dtype, hipStream_t s);
hipError_t launch_ssm_backward(const SsmArgs& a, int dtype, hipStream_t s);
size_t ssm_fold_bytes(const SsmArgs& a);
hipError_t launch_ssm_grad(const SsmArgs& a, int dtype, const float* ds, float* part, float* fold, hipStream_t s);

}  // namespace gdn
