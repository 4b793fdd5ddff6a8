// host_checks.h -- checks that the host entry points of gdn_layer.h and gdn_hybrid.h share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gdn.h"

namespace gdn {
namespace host {

constexpr size_t kAlign = 256;
// A launch holds less than 2^32 threads along x: 2^24 - 1 workgroups of up to 256.
constexpr int64_t kMaxBlocks = (1 << 24) - 1;

inline bool aligned(const void* ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

#define GDN_TRY(x)               \
  do {                           \
    const gdn_status s_ = (x);   \
    if (s_ != GDN_OK) return s_; \
  } while (0)

inline int esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// A row view that the call reads or writes (rows > 0).
inline gdn_status check_view(const void* ptr, int64_t rs, int64_t width, int dtype, int64_t rows) {
  if (rows == 0) return GDN_OK;
  if (!ptr || rs < width) return GDN_EINVAL;
  if (rs > INT64_MAX / 8 / (rows + 64)) return GDN_EINVAL;  // offsets stay within 64 bits
  if (!aligned(ptr, 16) || ((uint64_t)rs * esize(dtype)) % 16) return GDN_EALIGN;
  return GDN_OK;
}

inline gdn_status check_arr(const void* ptr, bool required, size_t align = 4) {
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
inline gdn_status check_in_place(int64_t rows, std::initializer_list<View> ins, std::initializer_list<View> outs) {
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
inline gdn_status check_apart(int64_t rows, std::initializer_list<const void*> ins, std::initializer_list<const void*> outs) {
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

inline gdn_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return GDN_OK;
  if (!ws || have < need) return GDN_EWORKSPACE;
  return aligned(ws, kAlign) ? GDN_OK : GDN_EALIGN;
}

inline gdn_status check_seqs(int N, int T, int64_t T_total, const void* cu) {
  if (N < 0 || T_total < 0) return GDN_EINVAL;
  if (!cu) {
    if (T < 0 || (int64_t)N * T != T_total) return GDN_EINVAL;
  } else if (N == 0 && T_total != 0) {
    return GDN_EINVAL;
  }
  if (T_total > (1 << 28)) return GDN_EINVAL;  // launch limits
  return aligned(cu, 4) ? GDN_OK : GDN_EALIGN;
}

inline gdn_status status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_EHIP; }

inline gdn_status check_slots(int N, int n_slots, const int32_t* idx) {
  if (n_slots < 0 || (!idx && n_slots < N)) return GDN_EINVAL;
  return check_arr(idx, false);
}

}  // namespace host
}  // namespace gdn
