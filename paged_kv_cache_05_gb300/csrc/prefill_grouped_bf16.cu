// The grouped kinds of the prompt-phase kernel, bf16.
#include "prefill_kernel.cuh"

cudaError_t pkv::launch_prefill_grouped_bf16(const CUtensorMap& tq, const CUtensorMap& tk,
                                      const CUtensorMap& tv, const PrefillArgs& a, int head_dim,
                                      int kind, cudaStream_t stream) {
    return head_dim == 128 ? launch_grouped<__nv_bfloat16, 128, 0>(tq, tk, tv, a, kind, stream)
                           : launch_grouped<__nv_bfloat16, 64, 0>(tq, tk, tv, a, kind, stream);
}
