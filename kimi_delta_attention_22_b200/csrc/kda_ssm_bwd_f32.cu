// kda_ssm_bwd_f32.cu -- the selective scan's gradients for fp32 activations.
#include "kda_ssm_bwd.cuh"

namespace kda {

cudaError_t launch_ssm_bwd_f32(const SsmArgs& a, cudaStream_t s) { return ssm::go_t<float>(a, s); }

}  // namespace kda
