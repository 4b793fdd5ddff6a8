// hybrid_internal.h -- descriptors shared by the host entry points of gdn_hybrid.h and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// glr.hip: everything of one forward, backward or token step of the gated linear recurrence.
struct GlrArgs {
  int N, T, ch;  // sequences, tokens per sequence when cu is null, channels
  int64_t rows;
  const int* cu;
  float rate;
  const float* lam;
  const int* fresh;
  const void *x, *r, *i, *dy;
  int64_t x_rs, r_rs, i_rs, dy_rs;
  const float *h0, *dhT;
  void *y, *dx, *dr, *di;
  int64_t y_rs, dx_rs, dr_rs, di_rs;
  float *hT, *dlam, *dh0;
  float* sv;     // states at the tiles' starts, or nullptr
  float* ws;
  float* state;  // decode: [n_slots][ch]
  int n_slots;
  const int* idx;
};
constexpr int kGlrTokenChannels = 128;  // of a workgroup of the token kernel
int64_t glr_blocks(const GlrArgs& a, int dtype);  // workgroups of a launch
size_t glr_fwd_ws_bytes(const GlrArgs& a, int dtype);
size_t glr_bwd_ws_bytes(const GlrArgs& a, int dtype);
size_t glr_saved_bytes(const GlrArgs& a);
hipError_t launch_glr_forward(const GlrArgs& a, int dtype, hipStream_t s);
hipError_t launch_glr_backward(const GlrArgs& a, int dtype, hipStream_t s);
hipError_t launch_glr_decode(const GlrArgs& a, int dtype, hipStream_t s);

// qk_rope.hip
struct RopeArgs {
  int64_t rows;
  int Hq, Hk, D, R, adjacent;
  float eps, scale;
  const int* pos;
  const double* freq;
  const float *wq, *wk;
  const void *q, *k, *v;   // backward: v is unused
  int64_t q_rs, k_rs, v_rs;
  const void *gq, *gk;     // backward: dqo, dko
  int64_t gq_rs, gk_rs;
  void *qo, *ko;           // or dq, dk
  int64_t qo_rs, ko_rs;
  void *kp, *vp;           // cache form: pages
  int page;
  int64_t places;          // n_pages * page
  const int* where;
  float *dwq, *dwk, *ws;
};
enum RopeKind { ROPE_FWD, ROPE_BWD, ROPE_CACHE };
size_t rope_bwd_ws_bytes(const RopeArgs& a);
hipError_t launch_rope(RopeKind kind, const RopeArgs& a, int dtype, hipStream_t s);

// paged_attn.hip
struct PagedArgs {
  int N, Hq, Hk, D, page, n_pages, max_pages, max_len, window;
  float scale;
  const int *table, *lens;
  const void *q, *kp, *vp;
  int64_t q_rs, out_rs;
  void* out;
  float* lse;
  float* ws;
};
int64_t paged_blocks(const PagedArgs& a, int dtype);  // workgroups of a launch
size_t paged_ws_bytes(const PagedArgs& a, int dtype);
hipError_t launch_paged(const PagedArgs& a, int dtype, hipStream_t s);

}  // namespace gdn
