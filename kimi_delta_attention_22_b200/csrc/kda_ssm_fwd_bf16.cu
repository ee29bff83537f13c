// kda_ssm_fwd_bf16.cu -- the selective scan for bf16 activations, and the size of the workspace
// (which does not depend on their type).
#include "kda_ssm_fwd.cuh"

namespace kda {

cudaError_t launch_ssm_fwd_f32(const SsmArgs& a, cudaStream_t s);   // kda_ssm_fwd_f32.cu

cudaError_t launch_ssm_fwd(const SsmArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? ssm::fwd_t<__nv_bfloat16>(a, s) : launch_ssm_fwd_f32(a, s);
}

size_t ssm_fwd_workspace_bytes(long long B, long long T, int D, int N, int G, bool varlen) {
    const ssm::Segments p = ssm::plan(B, T, D, N, G, varlen).seg;
    return p.whole ? 0 : sizeof(float) * (size_t)p.count * D * (N + 1);
}

}  // namespace kda
