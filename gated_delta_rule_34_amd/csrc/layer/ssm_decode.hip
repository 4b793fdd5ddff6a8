// ssm_decode.hip -- one step of the selective state space scan per sequence, on gfx950:
//
//   S' = a S + b (x) (D x),  y = S'^T c + d_skip x
//
// for every (row, head), the state of the row's slot updated in place. The state is read once and
// written once (8 Dk Dv bytes per row and head) and little else moves: bound by HBM. Plain VALU
// work in float32; the column sums of S' c are joined over the row groups in a fixed order. Measured:
// 256 rows x 64 heads of 128 x 64 take 185 us in a loop, 5.8 TB/s (a large copy reaches 5.2).
#include "vec8.h"

namespace gdn {

// Each thread owns 4 adjacent state columns of RPG rows rg + RG i, so that a wave reads whole
// consecutive rows.
template <int DK, int DV> struct SsmDecCfg {
  static constexpr int NT = DK * DV / 4 >= 256 ? 256 : DK * DV / 4;
  static constexpr int CPR = DV / 4, RG = NT / CPR, RPG = DK / RG;
  static_assert(RG * RPG == DK && NT % 64 == 0, "layout covers the state");
};

template <typename TI, int DK, int DV>
__global__ __launch_bounds__((SsmDecCfg<DK, DV>::NT)) void k_ssm_decode(SsmDecArgs a) {
  using CF = SsmDecCfg<DK, DV>;
  constexpr int NT = CF::NT, CPR = CF::CPR, RG = CF::RG, RPG = CF::RPG;
  __shared__ float sb[DK], sc[DK];
  __shared__ __align__(16) float part[RG][DV];
  const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv;
  const int slot = a.idx ? a.idx[n] : n;
  if (slot < 0 || slot >= a.n_slots) return;  // the row is skipped
  const int kh = h / a.r, t = threadIdx.x, c4 = (t % CPR) * 4, rg = t / CPR;
  float* S = a.state + ((int64_t)slot * a.Hv + h) * DK * DV;
  f32x4 s[RPG];
#pragma unroll
  for (int i = 0; i < RPG; ++i) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (rg + RG * i) * DV + c4));
  const TI* br = (const TI*)a.b + (int64_t)n * a.b_rs + kh * DK;
  const TI* cr = (const TI*)a.c + (int64_t)n * a.c_rs + kh * DK;
  for (int d = t; d < DK; d += NT) {
    sb[d] = (float)br[d];
    sc[d] = (float)cr[d];
  }
  const float z = a.dt[(int64_t)n * a.Hv + h] + (a.dt_bias ? a.dt_bias[h] : 0.f);
  const float step = softplusf(z), dec = expf(-decay_rate(a.a_log[h]) * step);
  const TI* xr = (const TI*)a.x + (int64_t)n * a.x_rs + h * DV + c4;
  const f32x4 x = {(float)xr[0], (float)xr[1], (float)xr[2], (float)xr[3]};
  const f32x4 u = step * x;
  __syncthreads();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int d = rg + RG * i;
    s[i] = dec * s[i] + sb[d] * u;
    __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + d * DV + c4));
    acc += sc[d] * s[i];
  }
  *reinterpret_cast<f32x4*>(&part[rg][c4]) = acc;
  __syncthreads();
  if (rg == 0) {
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < RG; ++j) y += *reinterpret_cast<const f32x4*>(&part[j][c4]);
    if (a.d_skip) y += a.d_skip[h] * x;
    TI* yr = (TI*)a.y + (int64_t)n * a.y_rs + h * DV + c4;
#pragma unroll
    for (int e = 0; e < 4; ++e) yr[e] = (TI)y[e];
  }
}

template <typename TI, int DK, int DV> static hipError_t dec_go(const SsmDecArgs& a, hipStream_t s) {
  traced("k_ssm_decode", s, [&] { k_ssm_decode<TI, DK, DV><<<a.N * a.Hv, SsmDecCfg<DK, DV>::NT, 0, s>>>(a); });
  return hipGetLastError();
}
template <typename TI, int DK> static hipError_t dec_v(const SsmDecArgs& a, hipStream_t s) {
  switch (a.Dv) {
    case 16: return dec_go<TI, DK, 16>(a, s);
    case 32: return dec_go<TI, DK, 32>(a, s);
    case 64: return dec_go<TI, DK, 64>(a, s);
    case 128: return dec_go<TI, DK, 128>(a, s);
  }
  return hipErrorInvalidValue;
}
template <typename TI> static hipError_t dec_k(const SsmDecArgs& a, hipStream_t s) {
  switch (a.Dk) {
    case 16: return dec_v<TI, 16>(a, s);
    case 32: return dec_v<TI, 32>(a, s);
    case 64: return dec_v<TI, 64>(a, s);
    case 128: return dec_v<TI, 128>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_ssm_decode(const SsmDecArgs& a, int dtype, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  return dtype == 0 ? dec_k<float>(a, s) : dec_k<__bf16>(a, s);
}

}  // namespace gdn
