// hybrid_host_stubs.cpp -- host-only stand-ins for the launchers and size queries of the other token
// mixers (hybrid_abi.cpp), as gdn_host_stubs.cpp has them for gdn_abi.cpp.
#include <hip/hip_runtime.h>

#include "hybrid/hybrid_internal.h"

namespace gdn {
int64_t glr_blocks(const GlrArgs& a, int) { return (a.rows / 512 + a.N) * ((a.ch + 31) / 32); }
size_t glr_fwd_ws_bytes(const GlrArgs&, int) { return 4096; }
size_t glr_bwd_ws_bytes(const GlrArgs&, int) { return 4096; }
size_t glr_saved_bytes(const GlrArgs&) { return 4096; }
hipError_t launch_glr_forward(const GlrArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_glr_backward(const GlrArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_glr_decode(const GlrArgs&, int, hipStream_t) { return hipSuccess; }
size_t rope_bwd_ws_bytes(const RopeArgs&) { return 4096; }
hipError_t launch_rope(RopeKind, const RopeArgs&, int, hipStream_t) { return hipSuccess; }
int64_t paged_blocks(const PagedArgs& a, int) { return (int64_t)a.N * a.Hk * (a.max_len / 128 + 1); }
size_t paged_ws_bytes(const PagedArgs&, int) { return 4096; }
hipError_t launch_paged(const PagedArgs&, int, hipStream_t) { return hipSuccess; }
}  // namespace gdn
