// vec8.h -- eight adjacent values of a row (one 16-byte bf16 piece, two float32 ones) as float32. In a
// namespace of its own: gdn_conv.hip has types of the same names, with another layout.
#pragma once
#include "../gdn_frag.h"
#include "../gdn_internal.h"
#include "layer_internal.h"

namespace gdn {
namespace layer {

struct F8 {
  float v[8];
};

template <typename TI> struct Raw8 {
  f32x4 a, b;
};
template <> struct Raw8<__bf16> {
  i32x4 a;
};

// Eight values as stored (converted at their use, so that a load in flight is not waited for).
// NT: non-temporal, for rows that are read once.
template <bool NT, typename TI> __device__ __forceinline__ Raw8<TI> ldraw8(const TI* p) {
  Raw8<TI> r;
  if constexpr (sizeof(TI) == 2) {
    const i32x4* q = reinterpret_cast<const i32x4*>(p);
    r.a = NT ? __builtin_nontemporal_load(q) : *q;
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(p);
    r.a = NT ? __builtin_nontemporal_load(q) : q[0];
    r.b = NT ? __builtin_nontemporal_load(q + 1) : q[1];
  }
  return r;
}

template <typename TI> __device__ __forceinline__ void straw8(TI* p, const Raw8<TI>& x) {
  if constexpr (sizeof(TI) == 2) {
    *reinterpret_cast<i32x4*>(p) = x.a;
  } else {
    *reinterpret_cast<f32x4*>(p) = x.a;
    *reinterpret_cast<f32x4*>(p + 4) = x.b;
  }
}

template <typename TI> __device__ __forceinline__ F8 cvt8(const Raw8<TI>& x) {
  F8 r;
  if constexpr (sizeof(TI) == 2) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, x.a);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = (float)b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = x.a[i];
      r.v[4 + i] = x.b[i];
    }
  }
  return r;
}

template <typename TI> __device__ __forceinline__ F8 ld8(const TI* p) { return cvt8<TI>(ldraw8<false, TI>(p)); }

template <typename TI> __device__ __forceinline__ void st8(TI* p, const F8& x) {
  if constexpr (sizeof(TI) == 2) {
    bf16x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (__bf16)x.v[i];
    *reinterpret_cast<bf16x8*>(p) = y;
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{x.v[0], x.v[1], x.v[2], x.v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{x.v[4], x.v[5], x.v[6], x.v[7]};
  }
}

// st8 past the caches' normal allocation, for results that nothing reads soon.
template <typename TI> __device__ __forceinline__ void st8nt(TI* p, const F8& x) {
  if constexpr (sizeof(TI) == 2) {
    bf16x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (__bf16)x.v[i];
    store_nt(reinterpret_cast<bf16x8*>(p), y);
  } else {
    store_nt(reinterpret_cast<f32x4*>(p), f32x4{x.v[0], x.v[1], x.v[2], x.v[3]});
    store_nt(reinterpret_cast<f32x4*>(p + 4), f32x4{x.v[4], x.v[5], x.v[6], x.v[7]});
  }
}

__device__ __forceinline__ F8 zero8() { return F8{{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}}; }

// 1 / (1 + e^-z); 0 where e^-z overflows, NaN for NaN. For float32 rows the exponential is within an ulp and
// the quotient rounded once. For bfloat16 rows both are the hardware's: e^-z is then some |z| 2^-24 off
// (its argument is rounded after the product with log2 e), 2^-17 at the most and far below a row's own 2^-8, and
// the accurate form would cost the streaming kernels a third (21488 rows x 10240 of the conv: 196 -> 265 us, float32:
// 9393 rows 189 -> 198).
template <typename TI> __device__ __forceinline__ float sigmoidf(float z) {
  if constexpr (sizeof(TI) == 2) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}

// The step of the scan: softplus(z), z itself past 20 (where they agree to float32).
__device__ __forceinline__ float softplusf(float z) { return z > 20.f ? z : log1pf(expf(z)); }

// exp(a_log), kept finite: a rate of 2^100 already leaves nothing of a state unless the step is zero, and
// then the decay is one (an infinite rate times a zero step would be NaN). NaN stays.
__device__ __forceinline__ float decay_rate(float a_log) {
  const float a = expf(a_log);
  return a > 0x1p100f ? 0x1p100f : a;
}

}  // namespace layer
using namespace layer;
}  // namespace gdn
