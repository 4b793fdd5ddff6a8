// rows.h -- rows of a caller's tensor through buffer resources: what lies past their end reads as zeros and
// is not written, without a branch.
#pragma once
#include <hip/hip_runtime.h>

#include "../gdn_frag.h"
#include "vec8.h"

namespace gdn {

// Raw buffer resource over [base, base + bytes), base and bytes wave-uniform: loads at or past `bytes`
// give zeros and stores there are dropped, without a branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every resource (a tile's rows span less than 2^31 bytes)
template <bool NT> __device__ __forceinline__ i32x4 buf_ld16(__amdgpu_buffer_rsrc_t rs, uint32_t voff) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)voff, 0, NT ? 2 : 0));
}
template <bool NT> __device__ __forceinline__ void buf_st16(__amdgpu_buffer_rsrc_t rs, uint32_t voff, i32x4 v) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), rs, (int)voff, 0, NT ? 2 : 0);
}

}  // namespace gdn
