// Paged attention with bf16 elements (the kernel is in paged_attention.cuh).
#include "paged_attention.cuh"

namespace lbcsr {

size_t attention_workspace_bf16(int dim, int group, int sms) {
    return with_mma<__nv_bfloat16>(dim, group, [&](auto tile) { return workspace_of<decltype(tile)>(sms); });
}

cudaError_t launch_attention_bf16(const spmv_paged_attention_t &a, int sms, cudaStream_t stream) {
    return with_mma<__nv_bfloat16>(a.head_dim, a.q_heads / a.kv_heads,
                                  [&](auto tile) { return launch_attention<decltype(tile)>(a, sms, stream); });
}

}  // namespace lbcsr
