// kda_ssm_bwd_bf16.cu -- the selective scan's gradients for bf16 activations, and the layout of
// the workspace (which does not depend on their type).
#include "kda_ssm_bwd.cuh"

namespace kda {

cudaError_t launch_ssm_bwd_f32(const SsmArgs& a, cudaStream_t s);   // kda_ssm_bwd_f32.cu

cudaError_t launch_ssm_bwd(const SsmArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? ssm::go_t<__nv_bfloat16>(a, s) : launch_ssm_bwd_f32(a, s);
}

size_t ssm_bwd_workspace_bytes(long long B, long long T, int D, int N, int G) {
    return ssm::layout(B * T, D, N, G).bytes;
}

}  // namespace kda
