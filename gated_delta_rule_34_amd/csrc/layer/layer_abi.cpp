// layer_abi.cpp -- host side of the C ABI declared in include/gdn_layer.h: argument checks and
// kernel launches. No allocation, no synchronisation.
#include "gdn_layer.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "layer_internal.h"

namespace {

constexpr size_t kAlign = 256;
// A launch holds less than 2^32 threads along x: 2^24 - 1 workgroups of up to 256.
constexpr int64_t kMaxBlocks = (1 << 24) - 1;

bool aligned(const void* ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

#define GDN_TRY(x)               \
  do {                           \
    const gdn_status s_ = (x);   \
    if (s_ != GDN_OK) return s_; \
  } while (0)

int esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// A row view that the call reads or writes (rows > 0).
gdn_status check_view(const void* ptr, int64_t rs, int64_t width, int dtype, int64_t rows) {
  if (rows == 0) return GDN_OK;
  if (!ptr || rs < width) return GDN_EINVAL;
  if (rs > INT64_MAX / 8 / (rows + 64)) return GDN_EINVAL;  // offsets stay within 64 bits
  if (!aligned(ptr, 16) || ((uint64_t)rs * esize(dtype)) % 16) return GDN_EALIGN;
  return GDN_OK;
}

gdn_status check_arr(const void* ptr, bool required, size_t align = 4) {
  if (!ptr) return required ? GDN_EINVAL : GDN_OK;
  return aligned(ptr, align) ? GDN_OK : GDN_EALIGN;
}

// A row view among a call's arguments.
struct View {
  const void* p;
  int64_t rs;
};

// For calls whose threads read what they need of the inputs before they write the same places: an output may be
// an input's very view. At an input's address with another stride, its rows would be rows that other threads
// still read. Two outputs are never at one address.
gdn_status check_in_place(int64_t rows, std::initializer_list<View> ins, std::initializer_list<View> outs) {
  if (rows == 0) return GDN_OK;
  for (const View* o = outs.begin(); o != outs.end(); ++o) {
    if (!o->p) continue;
    for (const View& i : ins)
      if (o->p == i.p && o->rs != i.rs && rows > 1) return GDN_EINVAL;
    for (const View* q = outs.begin(); q != o; ++q)
      if (o->p == q->p) return GDN_EINVAL;
  }
  return GDN_OK;
}

// For calls whose workgroups read what others write: an output is at no input's address, nor at another output's.
gdn_status check_apart(int64_t rows, std::initializer_list<const void*> ins, std::initializer_list<const void*> outs) {
  if (rows == 0) return GDN_OK;
  for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void* i : ins)
      if (*o == i) return GDN_EINVAL;
    for (const void* const* q = outs.begin(); q != o; ++q)
      if (*o == *q) return GDN_EINVAL;
  }
  return GDN_OK;
}

gdn_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return GDN_OK;
  if (!ws || have < need) return GDN_EWORKSPACE;
  return aligned(ws, kAlign) ? GDN_OK : GDN_EALIGN;
}

gdn_status check_seqs(int N, int T, int64_t T_total, const void* cu) {
  if (N < 0 || T_total < 0) return GDN_EINVAL;
  if (!cu) {
    if (T < 0 || (int64_t)N * T != T_total) return GDN_EINVAL;
  } else if (N == 0 && T_total != 0) {
    return GDN_EINVAL;
  }
  if (T_total > (1 << 28)) return GDN_EINVAL;  // launch limits
  return aligned(cu, 4) ? GDN_OK : GDN_EALIGN;
}

gdn_status status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_EHIP; }

// ------------------------------------------------------------------ scan

bool size_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

gdn_status check_ssm(const gdn_ssm_problem* p) {
  if (!p) return GDN_EINVAL;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_EUNSUPPORTED;
  if (p->Hk <= 0 || p->Hv <= 0 || p->Hv % p->Hk || p->Dk <= 0 || p->Dv <= 0) return GDN_EINVAL;
  if (!size_ok(p->Dk) || !size_ok(p->Dv)) return GDN_EUNSUPPORTED;
  GDN_TRY(check_seqs(p->N, p->T, p->T_total, p->cu_seqlens));
  // one workgroup per (sequence, head, 64 columns), per (row, head) and per (chunk, group)
  constexpr int64_t most = kMaxBlocks / 2;  // (of up to 512 threads)
  const int64_t slabs = p->Dv > 64 ? 2 : 1, slots = p->T_total / 64 + p->N;
  if (((int64_t)p->N + 8) * p->Hv > most / slabs || slots > most / p->Hv) return GDN_EINVAL;
  GDN_TRY(check_arr(p->a_log, true));
  GDN_TRY(check_arr(p->dt_bias, false));
  return check_arr(p->d_skip, false);
}

gdn::SsmArgs ssm_args(const gdn_ssm_problem* p) {
  gdn::SsmArgs a{};
  a.N = p->N;
  a.Hk = p->Hk;
  a.Hv = p->Hv;
  a.r = p->Hv / p->Hk;
  a.Dk = p->Dk;
  a.Dv = p->Dv;
  a.T = p->cu_seqlens ? 0 : p->T;
  a.T_total = p->T_total;
  a.cu = p->cu_seqlens;
  a.a_log = p->a_log;
  a.dt_bias = p->dt_bias;
  a.d_skip = p->d_skip;
  return a;
}

// A row view of the scan: its kernels address the 64 rows of a chunk with 31-bit byte offsets.
gdn_status ssm_view(const void* v, int64_t rs, int64_t width, int dtype, int64_t rows) {
  // 64 rows of 2^23 - 1 float32 values span less than 2^31 bytes
  if (rows > 0 && rs * esize(dtype) >= (int64_t)1 << 25) return GDN_EINVAL;
  return check_view(v, rs, width, dtype, rows);
}

// The views x, b, c and dt that every scan call reads.
gdn_status ssm_inputs(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                      const void* c, int64_t c_rs, const float* dt, gdn::SsmArgs& a) {
  const int64_t xw = (int64_t)p->Hv * p->Dv, kw = (int64_t)p->Hk * p->Dk;
  GDN_TRY(ssm_view(x, x_rs, xw, p->dtype, p->T_total));
  GDN_TRY(ssm_view(b, b_rs, kw, p->dtype, p->T_total));
  GDN_TRY(ssm_view(c, c_rs, kw, p->dtype, p->T_total));
  GDN_TRY(check_arr(dt, p->T_total > 0));
  a.x = x; a.x_rs = x_rs; a.b = b; a.b_rs = b_rs; a.c = c; a.c_rs = c_rs; a.dt = dt;
  return GDN_OK;
}

gdn_status check_slots(int N, int n_slots, const int32_t* idx) {
  if (n_slots < 0 || (!idx && n_slots < N)) return GDN_EINVAL;
  return check_arr(idx, false);
}

// ------------------------------------------------------------------ conv

gdn_status check_conv(const gdn_conv_problem* p) {
  if (!p || p->channels <= 0 || p->channels % 8) return GDN_EINVAL;
  if (p->kernel_size < 1 || p->kernel_size > 4) return GDN_EUNSUPPORTED;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_EUNSUPPORTED;
  if (p->channels / 8 > 65535LL * 64 || p->N > kMaxBlocks / 2) return GDN_EINVAL;  // grid limits
  GDN_TRY(check_seqs(p->N, p->T, p->T_total, p->cu_seqlens));
  // one wave per 512 channels of 64 rows and of each sequence's last rows
  const int64_t waves = (p->T_total / 64 + 64 + p->N) * ((p->channels + 511) / 512);
  return waves < (1LL << 32) / 64 ? GDN_OK : GDN_EINVAL;
}

gdn::ConvCarryArgs conv_args(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w,
                             const float* bias, void* y, int64_t y_rs) {
  gdn::ConvCarryArgs a{};
  a.N = p->N;
  a.T = p->cu_seqlens ? 0 : p->T;
  a.ch = p->channels;
  a.K = p->kernel_size;
  a.rows = p->T_total;
  a.cu = p->cu_seqlens;
  a.w = w;
  a.bias = bias;
  a.x = x;
  a.x_rs = x_rs;
  a.y = y;
  a.y_rs = y_rs;
  return a;
}

gdn_status conv_views(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w, const float* bias,
                      const void* y, int64_t y_rs) {
  GDN_TRY(check_view(x, x_rs, p->channels, p->dtype, p->T_total));
  GDN_TRY(check_view(y, y_rs, p->channels, p->dtype, p->T_total));
  GDN_TRY(check_arr(w, p->T_total > 0));
  return check_arr(bias, false);
}

// ------------------------------------------------------------------ norms

gdn_status check_norm(const gdn_norm_problem* p, bool add) {
  if (!p || p->rows < 0 || p->groups <= 0 || p->width <= 0 || p->width % 8) return GDN_EINVAL;
  if (p->width > 16384) return GDN_EUNSUPPORTED;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_EUNSUPPORTED;
  if (p->rows > INT32_MAX / p->groups || (int64_t)p->groups * p->width > INT32_MAX / 4) return GDN_EINVAL;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return GDN_EINVAL;
  if (add && (p->groups != 1 || !std::isfinite(p->scale))) return GDN_EINVAL;
  return GDN_OK;
}

gdn::NormArgs norm_args(const gdn_norm_problem* p) {
  gdn::NormArgs a{};
  a.rows = p->rows;
  a.groups = p->groups;
  a.width = p->width;
  a.shared = p->shared != 0;
  a.gate_first = p->gate_first != 0;
  a.eps = p->eps;
  a.scale = p->scale;
  return a;
}

gdn_status norm_view(const gdn_norm_problem* p, const void* v, int64_t rs) {
  return check_view(v, rs, (int64_t)p->groups * p->width, p->dtype, p->rows);
}

}  // namespace

extern "C" {

size_t gdn_ssm_fwd_workspace_bytes(const gdn_ssm_problem* p) {
  return check_ssm(p) == GDN_OK ? gdn::ssm_fwd_ws_bytes(ssm_args(p)) : 0;
}
size_t gdn_ssm_bwd_workspace_bytes(const gdn_ssm_problem* p) {
  return check_ssm(p) == GDN_OK ? gdn::ssm_bwd_ws_bytes(ssm_args(p)) : 0;
}
size_t gdn_ssm_chunk_state_bytes(const gdn_ssm_problem* p) {
  return check_ssm(p) == GDN_OK ? gdn::ssm_saved_bytes(ssm_args(p)) : 0;
}

gdn_status gdn_ssm_fwd(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                       const void* c, int64_t c_rs, const float* dt, const float* S0, void* y, int64_t y_rs,
                       float* S_T, void* chunk_states, void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_ssm(p));
  gdn::SsmArgs a = ssm_args(p);
  GDN_TRY(ssm_inputs(p, x, x_rs, b, b_rs, c, c_rs, dt, a));
  GDN_TRY(ssm_view(y, y_rs, (int64_t)p->Hv * p->Dv, p->dtype, p->T_total));
  GDN_TRY(check_apart(p->T_total, {x, b, c}, {y}));
  GDN_TRY(check_arr(S0, false, 16));
  GDN_TRY(check_arr(S_T, false, 16));
  if (S0 && S0 == S_T) return GDN_EINVAL;
  GDN_TRY(check_arr(chunk_states, false, 16));
  GDN_TRY(check_ws(workspace, workspace_bytes, gdn::ssm_fwd_ws_bytes(a)));
  if (p->N == 0) return GDN_OK;
  a.y = y; a.y_rs = y_rs; a.S0 = S0; a.ST = S_T;
  a.sv = static_cast<float*>(chunk_states);
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_ssm_forward(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_ssm_bwd(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                       const void* c, int64_t c_rs, const float* dt, const void* chunk_states,
                       const void* dy, int64_t dy_rs, const float* dS_T, void* dx, int64_t dx_rs, void* db,
                       int64_t db_rs, void* dc, int64_t dc_rs, float* ddt, float* da_log, float* ddt_bias,
                       float* dd_skip, float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_ssm(p));
  gdn::SsmArgs a = ssm_args(p);
  GDN_TRY(ssm_inputs(p, x, x_rs, b, b_rs, c, c_rs, dt, a));
  const int64_t xw = (int64_t)p->Hv * p->Dv, kw = (int64_t)p->Hk * p->Dk;
  GDN_TRY(ssm_view(dy, dy_rs, xw, p->dtype, p->T_total));
  GDN_TRY(ssm_view(dx, dx_rs, xw, p->dtype, p->T_total));
  GDN_TRY(ssm_view(db, db_rs, kw, p->dtype, p->T_total));
  GDN_TRY(ssm_view(dc, dc_rs, kw, p->dtype, p->T_total));
  // dx is written before x and dy are read for the last time, db and dc while other chunks' groups read theirs
  GDN_TRY(check_apart(p->T_total, {x, b, c, dy}, {dx}));
  GDN_TRY(check_apart(p->T_total, {x, b, c, dy}, {db}));
  GDN_TRY(check_apart(p->T_total, {x, b, c, dy}, {dc}));
  if (p->T_total > 0 && ddt == dt) return GDN_EINVAL;
  GDN_TRY(check_arr(ddt, p->T_total > 0));
  GDN_TRY(check_arr(da_log, false));
  GDN_TRY(check_arr(ddt_bias, false));
  GDN_TRY(check_arr(dd_skip, false));
  GDN_TRY(check_arr(dS_T, false, 16));
  GDN_TRY(check_arr(dS0, false, 16));
  if (dS_T && dS_T == dS0) return GDN_EINVAL;
  GDN_TRY(check_arr(chunk_states, p->T_total > 0, 16));
  GDN_TRY(check_ws(workspace, workspace_bytes, gdn::ssm_bwd_ws_bytes(a)));
  GDN_TRY(check_apart(p->T_total, {}, {dx, db, dc}));
  a.dy = dy; a.dy_rs = dy_rs; a.dST = dS_T;
  a.dx = dx; a.dx_rs = dx_rs; a.db = db; a.db_rs = db_rs; a.dc = dc; a.dc_rs = dc_rs;
  a.ddt = ddt; a.da_log = da_log; a.ddt_bias = ddt_bias; a.dd_skip = dd_skip; a.dS0 = dS0;
  a.sv = static_cast<float*>(const_cast<void*>(chunk_states));
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_ssm_backward(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_ssm_decode(const gdn_ssm_problem* p, const void* x, int64_t x_rs, const void* b, int64_t b_rs,
                          const void* c, int64_t c_rs, const float* dt, float* state, int32_t n_slots,
                          const int32_t* slot_idx, void* y, int64_t y_rs, void* stream) {
  GDN_TRY(check_ssm(p));
  if (p->cu_seqlens || p->T != 1 || p->T_total != p->N) return GDN_EINVAL;
  gdn::SsmArgs v = ssm_args(p);
  GDN_TRY(ssm_inputs(p, x, x_rs, b, b_rs, c, c_rs, dt, v));
  GDN_TRY(check_view(y, y_rs, (int64_t)p->Hv * p->Dv, p->dtype, p->N));
  GDN_TRY(check_arr(state, p->N > 0, 16));
  GDN_TRY(check_slots(p->N, n_slots, slot_idx));
  GDN_TRY(check_apart(p->N, {b, c}, {y}));  // a row's other heads may still read them
  GDN_TRY(check_in_place(p->N, {{x, x_rs}}, {{y, y_rs}}));
  gdn::SsmDecArgs a{};
  a.N = p->N; a.Hv = p->Hv; a.r = p->Hv / p->Hk; a.Dk = p->Dk; a.Dv = p->Dv; a.n_slots = n_slots;
  a.x = x; a.b = b; a.c = c; a.x_rs = x_rs; a.b_rs = b_rs; a.c_rs = c_rs; a.y = y; a.y_rs = y_rs;
  a.dt = dt; a.a_log = p->a_log; a.dt_bias = p->dt_bias; a.d_skip = p->d_skip;
  a.state = state; a.idx = slot_idx;
  return status_of(gdn::launch_ssm_decode(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_conv1d_silu_prompt(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w,
                                  const float* bias, const void* first, void* y, int64_t y_rs, void* last,
                                  void* stream) {
  GDN_TRY(check_conv(p));
  GDN_TRY(conv_views(p, x, x_rs, w, bias, y, y_rs));
  GDN_TRY(check_arr(first, false, 16));
  GDN_TRY(check_arr(last, false, 16));
  // runs and sequences' ends are written by workgroups of their own
  GDN_TRY(check_apart(p->T_total, {x}, {y}));
  if (p->kernel_size > 1) {
    GDN_TRY(check_apart(p->N, {first}, {last}));
    GDN_TRY(check_apart(p->T_total, {x, first}, {y, last}));
  }
  gdn::ConvCarryArgs a = conv_args(p, x, x_rs, w, bias, y, y_rs);
  a.first = first;
  a.last = last;
  return status_of(gdn::launch_conv_prompt(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_conv1d_silu_decode(const gdn_conv_problem* p, const void* x, int64_t x_rs, const float* w,
                                  const float* bias, void* state, int32_t n_slots, const int32_t* slot_idx,
                                  void* y, int64_t y_rs, void* stream) {
  GDN_TRY(check_conv(p));
  if (p->cu_seqlens || p->T != 1 || p->T_total != p->N) return GDN_EINVAL;
  GDN_TRY(conv_views(p, x, x_rs, w, bias, y, y_rs));
  GDN_TRY(check_arr(state, p->N > 0 && p->kernel_size > 1, 16));
  GDN_TRY(check_slots(p->N, n_slots, slot_idx));
  GDN_TRY(check_in_place(p->N, {{x, x_rs}}, {{y, y_rs}}));
  if (p->kernel_size > 1) GDN_TRY(check_apart(p->N, {x, y}, {state}));
  gdn::ConvCarryArgs a = conv_args(p, x, x_rs, w, bias, y, y_rs);
  a.state = state;
  a.n_slots = n_slots;
  a.idx = slot_idx;
  return status_of(gdn::launch_conv_decode(a, p->dtype, static_cast<hipStream_t>(stream)));
}

size_t gdn_gated_norm_bwd_workspace_bytes(const gdn_norm_problem* p) {
  return check_norm(p, false) == GDN_OK ? gdn::norm_ws_bytes(norm_args(p), false) : 0;
}
size_t gdn_add_norm_bwd_workspace_bytes(const gdn_norm_problem* p) {
  return check_norm(p, true) == GDN_OK ? gdn::norm_ws_bytes(norm_args(p), true) : 0;
}

gdn_status gdn_gated_norm_fwd(const gdn_norm_problem* p, const void* x, int64_t x_rs, const void* z, int64_t z_rs,
                              const float* w, void* y, int64_t y_rs, void* stream) {
  GDN_TRY(check_norm(p, false));
  GDN_TRY(norm_view(p, x, x_rs));
  GDN_TRY(norm_view(p, z, z_rs));
  GDN_TRY(norm_view(p, y, y_rs));
  GDN_TRY(check_arr(w, true, 16));
  GDN_TRY(check_in_place(p->rows, {{x, x_rs}, {z, z_rs}}, {{y, y_rs}}));
  gdn::NormArgs a = norm_args(p);
  a.x = x; a.x_rs = x_rs; a.z = z; a.z_rs = z_rs; a.w = w; a.o = y; a.o_rs = y_rs;
  return status_of(gdn::launch_norm(gdn::GATE_FWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_gated_norm_bwd(const gdn_norm_problem* p, const void* x, int64_t x_rs, const void* z, int64_t z_rs,
                              const float* w, const void* dy, int64_t dy_rs, void* dx, int64_t dx_rs, void* dz,
                              int64_t dz_rs, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_norm(p, false));
  GDN_TRY(norm_view(p, x, x_rs));
  GDN_TRY(norm_view(p, z, z_rs));
  GDN_TRY(norm_view(p, dy, dy_rs));
  GDN_TRY(norm_view(p, dx, dx_rs));
  GDN_TRY(norm_view(p, dz, dz_rs));
  GDN_TRY(check_arr(w, true, 16));
  GDN_TRY(check_arr(dw, false));
  gdn::NormArgs a = norm_args(p);
  if (dw) GDN_TRY(check_ws(workspace, workspace_bytes, gdn::norm_ws_bytes(a, false)));
  GDN_TRY(check_in_place(p->rows, {{x, x_rs}, {z, z_rs}, {dy, dy_rs}}, {{dx, dx_rs}, {dz, dz_rs}}));
  a.x = x; a.x_rs = x_rs; a.z = z; a.z_rs = z_rs; a.w = w; a.g = dy; a.g_rs = dy_rs;
  a.o = dx; a.o_rs = dx_rs; a.o2 = dz; a.o2_rs = dz_rs; a.dw = dw;
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_norm(gdn::GATE_BWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_add_norm_fwd(const gdn_norm_problem* p, const void* h, int64_t h_rs, const void* y, int64_t y_rs,
                            const float* s, const float* w, void* res, int64_t res_rs, void* out, int64_t out_rs,
                            void* stream) {
  GDN_TRY(check_norm(p, true));
  GDN_TRY(norm_view(p, h, h_rs));
  GDN_TRY(norm_view(p, y, y_rs));
  GDN_TRY(norm_view(p, res, res_rs));
  GDN_TRY(norm_view(p, out, out_rs));
  GDN_TRY(check_arr(s, false, 16));
  GDN_TRY(check_arr(w, true, 16));
  GDN_TRY(check_in_place(p->rows, {{h, h_rs}, {y, y_rs}}, {{res, res_rs}, {out, out_rs}}));
  gdn::NormArgs a = norm_args(p);
  a.x = h; a.x_rs = h_rs; a.z = y; a.z_rs = y_rs; a.s = s; a.w = w;
  a.o = res; a.o_rs = res_rs; a.o2 = out; a.o2_rs = out_rs;
  return status_of(gdn::launch_norm(gdn::ADD_FWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_add_norm_bwd(const gdn_norm_problem* p, const void* res, int64_t res_rs, const void* y, int64_t y_rs,
                            const float* s, const float* w, const void* dout, int64_t dout_rs, const void* dres,
                            int64_t dres_rs, void* dh, int64_t dh_rs, void* dy, int64_t dy_rs, float* dw, float* ds,
                            void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_norm(p, true));
  GDN_TRY(norm_view(p, res, res_rs));
  if (ds) GDN_TRY(norm_view(p, y, y_rs));
  GDN_TRY(norm_view(p, dout, dout_rs));
  if (dres) GDN_TRY(norm_view(p, dres, dres_rs));
  GDN_TRY(norm_view(p, dh, dh_rs));
  if (dy) GDN_TRY(norm_view(p, dy, dy_rs));
  GDN_TRY(check_arr(s, false, 16));
  GDN_TRY(check_arr(w, true, 16));
  GDN_TRY(check_arr(dw, false));
  GDN_TRY(check_arr(ds, false));
  gdn::NormArgs a = norm_args(p);
  if (dw || ds) GDN_TRY(check_ws(workspace, workspace_bytes, gdn::norm_ws_bytes(a, true)));
  GDN_TRY(check_in_place(p->rows, {{res, res_rs}, {ds ? y : nullptr, y_rs}, {dout, dout_rs}, {dres, dres_rs}},
                         {{dh, dh_rs}, {dy, dy_rs}}));
  a.x = res; a.x_rs = res_rs; a.z = y; a.z_rs = y_rs; a.s = s; a.w = w;
  a.g = dout; a.g_rs = dout_rs; a.g2 = dres; a.g2_rs = dres_rs;
  a.o = dh; a.o_rs = dh_rs; a.o2 = dy; a.o2_rs = dy_rs; a.dw = dw; a.ds = ds;
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_norm(gdn::ADD_BWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
