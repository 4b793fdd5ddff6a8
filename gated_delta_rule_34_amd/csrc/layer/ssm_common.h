// ssm_common.h -- what the scan's sweep and gradient kernels share.
//
// The scan runs in chunks of 64 tokens on the matrix cores. With gamma the running sum of log2 a
// inside a chunk, G = c b^T and Gamma_ij = 2^(gamma_i - gamma_j) for i >= j:
//   y_i = sum_{j <= i} Gamma_ij G_ij D_j x_j + 2^gamma_i S^T c_i + d_skip x_i
//   S  <- 2^gamma_n S + sum_j 2^(gamma_n - gamma_j) D_j b_j (x) x_j
// and the backward's state adjoint dS (flowing into a chunk's end) mirrors it in reverse time:
//   dx_j = D_j (sum_{i >= j} Gamma_ij G_ij dy_i + 2^(gamma_n - gamma_j) dS^T b_j) + d_skip dy_j
//   dS <- 2^gamma_n dS + sum_i 2^gamma_i c_i (x) dy_i
// so one kernel does both (b and c, x and dy, the two decays and the places of D swapped).
#pragma once
#include "../gdn_common.h"
#include "rows.h"
#include "vec8.h"

namespace gdn {

constexpr int SC = 64;  // tokens per chunk
constexpr int SP = 64;  // columns of x per workgroup (a head's slab)

// Rows of Cn elements in LDS, 16 bytes apart from one another: reads of 16 rows at one column and the
// transposed reads of 4 rows fall in different banks, and the addresses of a lane's reads differ by
// constants (the permuted layouts of gdn_frag.h took some 25 registers more for them).
template <typename T, int Cn> struct PadRow {
  static constexpr int LD = Cn + 16 / (int)sizeof(T);
  static constexpr int size(int R) { return R * LD; }
  __device__ __forceinline__ static int at(int r, int c) { return r * LD + c; }
};

// bfloat16 terms that a float32 factor is split into as a matrix operand: three (24 bits) where
// the result is float32, two (16 bits) where it is a bfloat16 row. One term's rounding would be as
// large as the row's own, and larger where the row's terms cancel.
template <typename TI> constexpr int ssm_split() { return sizeof(TI) == 2 ? 3 : 1; }
template <typename TI> constexpr int out_split() { return sizeof(TI) == 2 ? 2 : 1; }

template <typename TI, int KS> using FragT = typename Mf<TI, KS>::frag;

// v (the KE values of a fragment) as NS fragments that add up to it.
template <typename TI, int KS, int NS> __device__ __forceinline__ void split_frag(const float (&v)[Mf<TI, KS>::KE], FragT<TI, KS> (&o)[NS]) {
  if constexpr (KS == 4) {
    o[0] = v[0];
  } else {
    typedef float fv __attribute__((ext_vector_type(Mf<TI, KS>::KE)));
    fv rest;
#pragma unroll
    for (int j = 0; j < Mf<TI, KS>::KE; ++j) rest[j] = v[j];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      o[k] = __builtin_convertvector(rest, FragT<TI, KS>);
      if (k + 1 < NS) rest -= __builtin_convertvector(o[k], fv);
    }
  }
}

// Fragment x (contraction over tokens, STD order) with token t's value multiplied by w[t].
template <typename TI, int KS, int NS>
__device__ __forceinline__ void scale_split(FragT<TI, KS> x, const float* w, int s, FragT<TI, KS> (&o)[NS]) {
  const int g = lane_id() >> 4;
  float v[Mf<TI, KS>::KE];
  if constexpr (KS == 4) {
    v[0] = x * w[4 * s + g];
  } else {
#pragma unroll
    for (int j = 0; j < Mf<TI, KS>::KE; j += 4) {
      const f32x4 ww = *reinterpret_cast<const f32x4*>(w + kidx<KS, STD>(s, g, j));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j + e] = (float)x[j + e] * ww[e];
    }
  }
  split_frag<TI, KS, NS>(v, o);
}

// Step s of a contraction over the rows of accumulator tiles (ACC order), split.
template <typename TI, int KS, int NS>
__device__ __forceinline__ void acc_split(const f32x4* t, int s, FragT<TI, KS> (&o)[NS]) {
  float v[Mf<TI, KS>::KE];
#pragma unroll
  for (int j = 0; j < Mf<TI, KS>::KE; ++j) {
    if constexpr (KS == 4) v[j] = t[s >> 2][s & 3];
    else if constexpr (KS == 16) v[j] = t[s][j];
    else v[j] = t[2 * s + (j >> 2)][j & 3];
  }
  split_frag<TI, KS, NS>(v, o);
}

// Sum over the four lanes that share l % 16, in each of them: the halves of the wave exchanged, then
// the halves of each half.
__device__ __forceinline__ float group4_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Four adjacent values of a row as float32, and back.
template <typename TI> __device__ __forceinline__ f32x4 ld4(const TI* p) {
  if constexpr (sizeof(TI) == 2) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
  } else {
    return *reinterpret_cast<const f32x4*>(p);
  }
}
template <typename TI> __device__ __forceinline__ void st4(TI* p, f32x4 v) {
  if constexpr (sizeof(TI) == 2)
    *reinterpret_cast<bf16x4*>(p) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  else
    *reinterpret_cast<f32x4*>(p) = v;
}

template <typename TI> __device__ __forceinline__ void buf_st4(__amdgpu_buffer_rsrc_t rs, uint32_t voff, f32x4 v) {
  if constexpr (sizeof(TI) == 2) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(
        __builtin_bit_cast(u2, bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]}), rs, (int)voff, 0, 0);
  } else {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), rs, (int)voff, 0, 0);
  }
}

// A [64][CN] tile of rows on its way through registers into LDS, by NT threads. Rows at or past
// len and columns at or past ncols arrive as zeros; nothing outside the caller's rows is read.
template <typename TI, int CN, class L, int NT> struct TileRegs {
  static constexpr int CE = 16 / (int)sizeof(TI), PPR = CN / CE, TOT = SC * PPR, U = (TOT + NT - 1) / NT, STEP = NT / PPR;
  i32x4 v[U];
  uint32_t rsb, voff;  // row stride in bytes, this thread's first piece
  __device__ __forceinline__ void init(int64_t rs, int ncols) {
    const int q = (int)threadIdx.x, c = (q % PPR) * CE;
    rsb = (uint32_t)rs * (uint32_t)sizeof(TI);
    voff = q < TOT && c < ncols ? (uint32_t)(q / PPR) * rsb + c * (int)sizeof(TI) : kNowhere;
  }
  template <bool ONCE> __device__ __forceinline__ void load(const TI* src, int len) {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(src, (uint32_t)len * rsb);
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = buf_ld16<ONCE>(rs, voff + (uint32_t)(u * STEP) * rsb);
  }
  __device__ __forceinline__ void store(TI* lds) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = u * NT + (int)threadIdx.x;
      if (TOT % NT == 0 || q < TOT) *reinterpret_cast<i32x4*>(lds + L::at(q / PPR, (q % PPR) * CE)) = v[u];
    }
  }
};

// Inclusive sum over lanes 0..l in 64 bits. The exponents gamma_i - gamma_j are small differences
// of sums that reach hundreds: they are kept as a float32 pair (value and remainder).
template <int CTRL, int ROWS = 0xF> __device__ __forceinline__ double dppd(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan_incl_f64(double x) {
  x += dppd<0x111>(x);       // row_shr:1
  x += dppd<0x112>(x);       // row_shr:2
  x += dppd<0x114>(x);       // row_shr:4
  x += dppd<0x118>(x);       // row_shr:8
  x += dppd<0x142, 0xA>(x);  // row_bcast:15
  x += dppd<0x143, 0xC>(x);  // row_bcast:31
  return x;
}
__device__ __forceinline__ double lane_value_f64(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// -exp(a_log) in log2 units. The float32 exponential's ulp (1e-7 of a_log, as in the elementary operations) is common
// to all decays of a head; nothing behind it is rounded again before the sums of the gates. (An exponential in
// 64 bits, be it a short series, costs the gradient kernel some 18 spilled registers more.)
__device__ __forceinline__ double neg_a_log2(float a_log) { return -(double)decay_rate(a_log) * 1.4426950408889634; }

// 2^x with the part of x that a float32 drops.
__device__ __forceinline__ float exp2_d(double x) {
  const float hi = (float)x, lo = (float)(x - (double)hi), e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.69314718f, e);
}

// Gates of one chunk, one token per lane: the step, gamma (log2), its sum over the chunk.
struct Gate {
  float z, step;
  double gam, tot;
};
__device__ __forceinline__ Gate chunk_gate(float dt, float bias, double neg_a, bool valid) {
  Gate q;
  q.z = dt + bias;
  q.step = valid ? softplusf(q.z) : 0.f;
  // One token's exponent ends at -4096: 2^-4096 is zero in every use, and a larger one would cost the
  // differences of its chunk's other tokens their accuracy (or, infinite, make them NaN).
  const double e = neg_a * (double)q.step;
  q.gam = wave_scan_incl_f64(valid ? (e < -4096.0 ? -4096.0 : e) : 0.0);
  q.tot = lane_value_f64(q.gam, 63);
  return q;
}

// Rows [lo, hi) of sequence n (wave-uniform), clamped into [0, T_total].
__device__ __forceinline__ void ssm_seq(const int* cu, int T, int64_t T_total, int n, int64_t& lo, int64_t& hi) {
  if (cu) {
    int64_t x = __builtin_amdgcn_readfirstlane(cu[n]), y = __builtin_amdgcn_readfirstlane(cu[n + 1]);
    x = x < 0 ? 0 : (x > T_total ? T_total : x);
    y = y < x ? x : (y > T_total ? T_total : y);
    lo = x;
    hi = y;
  } else {
    lo = (int64_t)n * T;
    hi = lo + T;
  }
}

// Slots of the per-chunk arrays without a table: chunk k of sequence n (rows [lo, hi)) has slot
// lo / 64 + n + k. A sequence of len rows has ceil(len / 64) <= hi / 64 - lo / 64 + 1 chunks, so
// no two chunks share a slot and all are below T_total / 64 + N.
__host__ __device__ __forceinline__ int64_t ssm_slots(int64_t T_total, int N) { return T_total / SC + N; }

}  // namespace gdn
