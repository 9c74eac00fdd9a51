// The grouped kinds of the prompt-phase kernel, fp16.
#include "prefill_kernel.cuh"

cudaError_t pkv::launch_prefill_grouped_f16(const CUtensorMap& tq, const CUtensorMap& tk,
                                      const CUtensorMap& tv, const PrefillArgs& a, int head_dim,
                                      int kind, cudaStream_t stream) {
    return head_dim == 128 ? launch_grouped<__half, 128, 0>(tq, tk, tv, a, kind, stream)
                           : launch_grouped<__half, 64, 0>(tq, tk, tv, a, kind, stream);
}
