// layer_host_stubs.cpp -- host-only stand-ins for the launchers and size queries of the layer's
// operators (layer_abi.cpp), as gdn_host_stubs.cpp has them for gdn_abi.cpp.
#include <hip/hip_runtime.h>

#include "layer/layer_internal.h"

namespace gdn {
hipError_t launch_conv_prompt(const ConvCarryArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_conv_decode(const ConvCarryArgs&, int, hipStream_t) { return hipSuccess; }
size_t norm_ws_bytes(const NormArgs&, bool) { return 4096; }
hipError_t launch_norm(NormKind, const NormArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ssm_decode(const SsmDecArgs&, int, hipStream_t) { return hipSuccess; }
size_t ssm_fwd_ws_bytes(const SsmArgs&) { return 4096; }
size_t ssm_bwd_ws_bytes(const SsmArgs&) { return 4096; }
size_t ssm_saved_bytes(const SsmArgs&) { return 4096; }
hipError_t launch_ssm_forward(const SsmArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ssm_backward(const SsmArgs&, int, hipStream_t) { return hipSuccess; }
}  // namespace gdn
