// kda_ssm_fwd_f32.cu -- the selective scan for fp32 activations.
#include "kda_ssm_fwd.cuh"

namespace kda {

cudaError_t launch_ssm_fwd_f32(const SsmArgs& a, cudaStream_t s) { return ssm::fwd_t<float>(a, s); }

}  // namespace kda
