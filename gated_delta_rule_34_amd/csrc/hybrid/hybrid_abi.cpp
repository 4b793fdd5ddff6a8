// hybrid_abi.cpp -- host side of the C ABI declared in include/gdn_hybrid.h: argument checks and
// kernel launches. No allocation, no synchronisation.
#include "gdn_hybrid.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../layer/host_checks.h"
#include "hybrid_internal.h"

using namespace gdn::host;

namespace {

bool known_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

// ------------------------------------------------------------------ gated linear recurrence

gdn::GlrArgs glr_args(const gdn_glr_problem* p) {
  gdn::GlrArgs a{};
  a.N = p->N;
  a.T = p->cu_seqlens ? 0 : p->T;
  a.ch = p->channels;
  a.rows = p->T_total;
  a.cu = p->cu_seqlens;
  a.rate = p->rate;
  a.lam = p->lambda;
  a.fresh = p->fresh;
  return a;
}

constexpr int64_t kGlrRowBytes = 1 << 23;

gdn_status check_glr(const gdn_glr_problem* p) {
  if (!p || p->channels <= 0 || p->channels % 8) return GDN_EINVAL;
  if (!known_dtype(p->dtype)) return GDN_EUNSUPPORTED;
  if (!std::isfinite(p->rate) || p->rate <= 0.f) return GDN_EINVAL;
  GDN_TRY(check_seqs(p->N, p->T, p->T_total, p->cu_seqlens));
  GDN_TRY(check_arr(p->lambda, true, 16));
  GDN_TRY(check_arr(p->fresh, false));
  // a row's stride is below 2^23 bytes (glr_view), and so are its channels, rows or none; the token kernel's grid then ends far below 65536
  if (p->channels >= kGlrRowBytes / esize(p->dtype)) return GDN_EINVAL;
  static_assert(kGlrRowBytes / 2 / gdn::kGlrTokenChannels < 65535, "grid.y of k_glr_decode");
  // launch limit: workgroups of 512 threads
  if (p->N > kMaxBlocks / 2) return GDN_EINVAL;
  return gdn::glr_blocks(glr_args(p), p->dtype) <= kMaxBlocks / 2 ? GDN_OK : GDN_EINVAL;
}

// A row view of the recurrence: its kernels address the rows of two tiles of 128 with 31-bit byte offsets.
gdn_status glr_view(const gdn_glr_problem* p, const void* v, int64_t rs) {
  if (p->T_total > 0 && rs >= kGlrRowBytes / esize(p->dtype)) return GDN_EINVAL;
  return check_view(v, rs, p->channels, p->dtype, p->T_total);
}

gdn_status glr_inputs(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs, const void* i,
                      int64_t i_rs, gdn::GlrArgs& a) {
  GDN_TRY(glr_view(p, x, x_rs));
  GDN_TRY(glr_view(p, r, r_rs));
  GDN_TRY(glr_view(p, i, i_rs));
  a.x = x; a.x_rs = x_rs; a.r = r; a.r_rs = r_rs; a.i = i; a.i_rs = i_rs;
  return GDN_OK;
}

// ------------------------------------------------------------------ norm and rotation

gdn_status check_rope(const gdn_qk_rope_problem* p) {
  if (!p || p->rows < 0 || p->Hq <= 0 || p->Hk <= 0 || p->D <= 0 || p->rot < 0 || p->rot > p->D) return GDN_EINVAL;
  if (!known_dtype(p->dtype) || p->D > 256 || p->D % 16 || p->rot % 16) return GDN_EUNSUPPORTED;
  const int64_t heads = (int64_t)p->Hq + 2 * (int64_t)p->Hk;
  if (heads > INT32_MAX / 1024 || p->rows > INT32_MAX / heads || p->rows > kMaxBlocks * 2) return GDN_EINVAL;
  if (!std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->rope_scale)) return GDN_EINVAL;
  const bool turned = p->rot > 0 && p->rows > 0;
  GDN_TRY(check_arr(p->positions, turned));
  GDN_TRY(check_arr(p->freq, turned, 8));
  GDN_TRY(check_arr(p->wq, false, 16));
  return check_arr(p->wk, false, 16);
}

gdn::RopeArgs rope_args(const gdn_qk_rope_problem* p) {
  gdn::RopeArgs a{};
  a.rows = p->rows;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.D = p->D;
  a.R = p->rot;
  a.adjacent = p->adjacent != 0;
  a.eps = p->eps;
  a.scale = p->rope_scale;
  a.pos = p->positions;
  a.freq = p->freq;
  a.wq = p->wq;
  a.wk = p->wk;
  return a;
}

gdn_status rope_view(const gdn_qk_rope_problem* p, const void* v, int64_t rs, int heads) {
  return check_view(v, rs, (int64_t)heads * p->D, p->dtype, p->rows);
}

// ------------------------------------------------------------------ paged attention

// A pool's places and the rows of its heads are counted in 31 and 32 bits.
gdn_status check_pool(int64_t n_pages, int64_t page_size, int64_t Hk) {
  if (n_pages < 0 || page_size < 1) return GDN_EINVAL;
  if (n_pages > INT32_MAX / page_size || n_pages * page_size > UINT32_MAX / Hk) return GDN_EINVAL;
  return GDN_OK;
}

gdn::PagedArgs paged_args(const gdn_paged_problem* p) {
  gdn::PagedArgs a{};
  a.N = p->N;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.D = p->D;
  a.page = p->page_size;
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.max_len = p->max_len;
  a.window = p->window;
  a.scale = p->scale;
  a.table = p->page_table;
  a.lens = p->lens;
  return a;
}

gdn_status check_paged(const gdn_paged_problem* p) {
  if (!p || p->N < 0 || p->Hq <= 0 || p->Hk <= 0 || p->Hq % p->Hk) return GDN_EINVAL;
  if (!known_dtype(p->dtype) || (p->D != 32 && p->D != 64 && p->D != 128 && p->D != 256)) return GDN_EUNSUPPORTED;
  GDN_TRY(check_pool(p->n_pages, p->page_size, p->Hk));
  if (p->max_pages < 0 || p->max_pages > INT32_MAX / p->page_size) return GDN_EINVAL;
  if (p->max_len < 0 || p->max_len > p->max_pages * p->page_size || p->window < 0 || !std::isfinite(p->scale)) return GDN_EINVAL;
  if (p->max_len > 1 << 30) return GDN_EINVAL;  // tokens past a chunk's end are counted in 31 bits too
  // launch limits: a workgroup per query head and sequence, and per chunk of a key head
  if ((int64_t)p->N * p->Hq > kMaxBlocks || gdn::paged_blocks(paged_args(p), p->dtype) > kMaxBlocks) return GDN_EINVAL;
  GDN_TRY(check_arr(p->page_table, p->N > 0 && p->max_len > 0));
  return check_arr(p->lens, p->N > 0);
}

}  // namespace

extern "C" {

size_t gdn_glr_fwd_workspace_bytes(const gdn_glr_problem* p) {
  return check_glr(p) == GDN_OK ? gdn::glr_fwd_ws_bytes(glr_args(p), p->dtype) : 0;
}
size_t gdn_glr_bwd_workspace_bytes(const gdn_glr_problem* p) {
  return check_glr(p) == GDN_OK ? gdn::glr_bwd_ws_bytes(glr_args(p), p->dtype) : 0;
}
size_t gdn_glr_state_bytes(const gdn_glr_problem* p) { return check_glr(p) == GDN_OK ? gdn::glr_saved_bytes(glr_args(p)) : 0; }

gdn_status gdn_glr_fwd(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                       const void* i, int64_t i_rs, const float* h0, void* y, int64_t y_rs, float* h_T,
                       void* states, void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_glr(p));
  gdn::GlrArgs a = glr_args(p);
  GDN_TRY(glr_inputs(p, x, x_rs, r, r_rs, i, i_rs, a));
  GDN_TRY(glr_view(p, y, y_rs));
  GDN_TRY(check_in_place(p->T_total, {{x, x_rs}, {r, r_rs}, {i, i_rs}}, {{y, y_rs}}));
  GDN_TRY(check_arr(h0, false, 16));
  GDN_TRY(check_arr(h_T, false, 16));
  if (h0 && h0 == h_T) return GDN_EINVAL;
  GDN_TRY(check_arr(states, false, 16));
  GDN_TRY(check_ws(workspace, workspace_bytes, gdn::glr_fwd_ws_bytes(a, p->dtype)));
  a.h0 = h0; a.y = y; a.y_rs = y_rs; a.hT = h_T;
  a.sv = static_cast<float*>(states);
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_glr_forward(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_glr_bwd(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                       const void* i, int64_t i_rs, const void* states, const void* dy, int64_t dy_rs,
                       const float* dh_T, void* dx, int64_t dx_rs, void* dr, int64_t dr_rs, void* di,
                       int64_t di_rs, float* dlambda, float* dh0, void* workspace, size_t workspace_bytes,
                       void* stream) {
  GDN_TRY(check_glr(p));
  gdn::GlrArgs a = glr_args(p);
  GDN_TRY(glr_inputs(p, x, x_rs, r, r_rs, i, i_rs, a));
  GDN_TRY(glr_view(p, dy, dy_rs));
  GDN_TRY(glr_view(p, dx, dx_rs));
  GDN_TRY(glr_view(p, dr, dr_rs));
  GDN_TRY(glr_view(p, di, di_rs));
  GDN_TRY(check_in_place(p->T_total, {{x, x_rs}, {r, r_rs}, {i, i_rs}, {dy, dy_rs}}, {{dx, dx_rs}, {dr, dr_rs}, {di, di_rs}}));
  GDN_TRY(check_arr(dh_T, false, 16));
  GDN_TRY(check_arr(dh0, false, 16));
  GDN_TRY(check_arr(dlambda, false));
  if (dh_T && dh_T == dh0) return GDN_EINVAL;
  GDN_TRY(check_arr(states, p->T_total > 0, 16));
  // the parts of dlambda, and the segments' maps
  GDN_TRY(check_ws(workspace, workspace_bytes, gdn::glr_bwd_ws_bytes(a, p->dtype)));
  a.sv = static_cast<float*>(const_cast<void*>(states));
  a.dy = dy; a.dy_rs = dy_rs; a.dhT = dh_T;
  a.dx = dx; a.dx_rs = dx_rs; a.dr = dr; a.dr_rs = dr_rs; a.di = di; a.di_rs = di_rs; a.dlam = dlambda; a.dh0 = dh0;
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_glr_backward(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_glr_decode(const gdn_glr_problem* p, const void* x, int64_t x_rs, const void* r, int64_t r_rs,
                          const void* i, int64_t i_rs, float* state, int32_t n_slots, const int32_t* slot_idx,
                          void* y, int64_t y_rs, void* stream) {
  GDN_TRY(check_glr(p));
  if (p->cu_seqlens || p->T != 1 || p->T_total != p->N) return GDN_EINVAL;
  gdn::GlrArgs a = glr_args(p);
  GDN_TRY(glr_inputs(p, x, x_rs, r, r_rs, i, i_rs, a));
  GDN_TRY(check_view(y, y_rs, p->channels, p->dtype, p->N));
  GDN_TRY(check_arr(state, p->N > 0, 16));
  GDN_TRY(check_slots(p->N, n_slots, slot_idx));
  GDN_TRY(check_in_place(p->N, {{x, x_rs}, {r, r_rs}, {i, i_rs}}, {{y, y_rs}}));
  GDN_TRY(check_apart(p->N, {x, r, i, y}, {state}));
  a.y = y; a.y_rs = y_rs; a.state = state; a.n_slots = n_slots; a.idx = slot_idx;
  return status_of(gdn::launch_glr_decode(a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_qk_rope_fwd(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                           void* qo, int64_t qo_rs, void* ko, int64_t ko_rs, void* stream) {
  GDN_TRY(check_rope(p));
  GDN_TRY(rope_view(p, q, q_rs, p->Hq));
  GDN_TRY(rope_view(p, k, k_rs, p->Hk));
  GDN_TRY(rope_view(p, qo, qo_rs, p->Hq));
  GDN_TRY(rope_view(p, ko, ko_rs, p->Hk));
  GDN_TRY(check_apart(p->rows, {k}, {qo}));
  GDN_TRY(check_apart(p->rows, {q}, {ko}));
  GDN_TRY(check_in_place(p->rows, {{q, q_rs}, {k, k_rs}}, {{qo, qo_rs}, {ko, ko_rs}}));
  gdn::RopeArgs a = rope_args(p);
  a.q = q; a.q_rs = q_rs; a.k = k; a.k_rs = k_rs; a.qo = qo; a.qo_rs = qo_rs; a.ko = ko; a.ko_rs = ko_rs;
  return status_of(gdn::launch_rope(gdn::ROPE_FWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

size_t gdn_qk_rope_bwd_workspace_bytes(const gdn_qk_rope_problem* p) {
  return check_rope(p) == GDN_OK ? gdn::rope_bwd_ws_bytes(rope_args(p)) : 0;
}

gdn_status gdn_qk_rope_bwd(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                           const void* dqo, int64_t dqo_rs, const void* dko, int64_t dko_rs, void* dq, int64_t dq_rs,
                           void* dk, int64_t dk_rs, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                           void* stream) {
  GDN_TRY(check_rope(p));
  GDN_TRY(rope_view(p, q, q_rs, p->Hq));
  GDN_TRY(rope_view(p, k, k_rs, p->Hk));
  GDN_TRY(rope_view(p, dqo, dqo_rs, p->Hq));
  GDN_TRY(rope_view(p, dko, dko_rs, p->Hk));
  GDN_TRY(rope_view(p, dq, dq_rs, p->Hq));
  GDN_TRY(rope_view(p, dk, dk_rs, p->Hk));
  GDN_TRY(check_apart(p->rows, {k, dko}, {dq}));
  GDN_TRY(check_apart(p->rows, {q, dqo}, {dk}));
  GDN_TRY(check_in_place(p->rows, {{q, q_rs}, {k, k_rs}, {dqo, dqo_rs}, {dko, dko_rs}}, {{dq, dq_rs}, {dk, dk_rs}}));
  GDN_TRY(check_arr(dwq, false));
  GDN_TRY(check_arr(dwk, false));
  if (dwq && dwq == dwk) return GDN_EINVAL;
  gdn::RopeArgs a = rope_args(p);
  if (dwq || dwk) GDN_TRY(check_ws(workspace, workspace_bytes, gdn::rope_bwd_ws_bytes(a)));
  a.q = q; a.q_rs = q_rs; a.k = k; a.k_rs = k_rs; a.gq = dqo; a.gq_rs = dqo_rs; a.gk = dko; a.gk_rs = dko_rs;
  a.qo = dq; a.qo_rs = dq_rs; a.ko = dk; a.ko_rs = dk_rs; a.dwq = dwq; a.dwk = dwk;
  a.ws = dwq || dwk ? static_cast<float*>(workspace) : nullptr;
  return status_of(gdn::launch_rope(gdn::ROPE_BWD, a, p->dtype, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_qk_rope_cache(const gdn_qk_rope_problem* p, const void* q, int64_t q_rs, const void* k, int64_t k_rs,
                             const void* v, int64_t v_rs, void* qo, int64_t qo_rs, void* k_pages, void* v_pages,
                             int32_t n_pages, int32_t page_size, const int32_t* where, void* stream) {
  GDN_TRY(check_rope(p));
  GDN_TRY(check_pool(n_pages, page_size, p->Hk));
  GDN_TRY(rope_view(p, q, q_rs, p->Hq));
  GDN_TRY(rope_view(p, k, k_rs, p->Hk));
  GDN_TRY(rope_view(p, v, v_rs, p->Hk));
  GDN_TRY(rope_view(p, qo, qo_rs, p->Hq));
  const bool pool = p->rows > 0 && n_pages > 0;
  GDN_TRY(check_arr(k_pages, pool, 16));
  GDN_TRY(check_arr(v_pages, pool, 16));
  GDN_TRY(check_arr(where, p->rows > 0));
  GDN_TRY(check_apart(p->rows, {k, v}, {qo}));
  GDN_TRY(check_apart(p->rows, {q, k, v, qo}, {k_pages, v_pages}));
  GDN_TRY(check_in_place(p->rows, {{q, q_rs}}, {{qo, qo_rs}}));
  gdn::RopeArgs a = rope_args(p);
  a.q = q; a.q_rs = q_rs; a.k = k; a.k_rs = k_rs; a.v = v; a.v_rs = v_rs; a.qo = qo; a.qo_rs = qo_rs;
  a.kp = k_pages; a.vp = v_pages; a.page = page_size; a.places = (int64_t)n_pages * page_size; a.where = where;
  return status_of(gdn::launch_rope(gdn::ROPE_CACHE, a, p->dtype, static_cast<hipStream_t>(stream)));
}

size_t gdn_paged_attn_workspace_bytes(const gdn_paged_problem* p) {
  return check_paged(p) == GDN_OK ? gdn::paged_ws_bytes(paged_args(p), p->dtype) : 0;
}

gdn_status gdn_paged_attn_decode(const gdn_paged_problem* p, const void* q, int64_t q_rs, const void* k_pages,
                                 const void* v_pages, void* out, int64_t out_rs, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  GDN_TRY(check_paged(p));
  const int64_t width = (int64_t)p->Hq * p->D;
  GDN_TRY(check_view(q, q_rs, width, p->dtype, p->N));
  GDN_TRY(check_view(out, out_rs, width, p->dtype, p->N));
  const bool pool = p->N > 0 && p->n_pages > 0 && p->max_len > 0;
  GDN_TRY(check_arr(k_pages, pool, 16));
  GDN_TRY(check_arr(v_pages, pool, 16));
  GDN_TRY(check_arr(lse, false));
  GDN_TRY(check_apart(p->N, {q, k_pages, v_pages}, {out}));
  gdn::PagedArgs a = paged_args(p);
  GDN_TRY(check_ws(workspace, workspace_bytes, gdn::paged_ws_bytes(a, p->dtype)));
  a.q = q; a.q_rs = q_rs; a.kp = k_pages; a.vp = v_pages; a.out = out; a.out_rs = out_rs; a.lse = lse;
  a.ws = static_cast<float*>(workspace);
  return status_of(gdn::launch_paged(a, p->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
