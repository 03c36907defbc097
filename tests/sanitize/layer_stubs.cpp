// Stand-ins for the launchers behind kda_layer_abi.cpp, so that its argument checks, workspace
// layout and plan of the scan's segments can be built with the host compiler under
// AddressSanitizer and UndefinedBehaviorSanitizer.  Each keeps the parameters it was given.
#include <hip/hip_runtime_api.h>

#include "../../gated_delta_rule_log2_amd/csrc/kda_layer.h"

int g_stub_launches = 0;
kda::SsmParams g_ssm;

namespace kda {
int conv_bwd_blocks(const ConvParams &p) { return p.tokens > 0 ? (int)((p.tokens + 63) / 64) : 0; }
int norm_bwd_blocks(const NormParams &p) { return p.rows < 768 ? (int)p.rows : 768; }
hipError_t launch_conv_fwd(const ConvParams &, hipStream_t) { ++g_stub_launches; return hipSuccess; }
hipError_t launch_conv_bwd(const ConvParams &, hipStream_t) { ++g_stub_launches; return hipSuccess; }
hipError_t launch_conv_step(const ConvParams &, hipStream_t) { ++g_stub_launches; return hipSuccess; }
hipError_t launch_norm_fwd(const NormParams &, bool, hipStream_t) { ++g_stub_launches; return hipSuccess; }
hipError_t launch_norm_bwd(const NormParams &, hipStream_t) { ++g_stub_launches; return hipSuccess; }
hipError_t launch_ssm_fwd(const SsmParams &p, hipStream_t) { ++g_stub_launches; g_ssm = p; return hipSuccess; }
hipError_t launch_ssm_bwd(const SsmParams &p, hipStream_t) { ++g_stub_launches; g_ssm = p; return hipSuccess; }
hipError_t launch_ssm_step(const SsmParams &p, hipStream_t) { ++g_stub_launches; g_ssm = p; return hipSuccess; }
}  // namespace kda
