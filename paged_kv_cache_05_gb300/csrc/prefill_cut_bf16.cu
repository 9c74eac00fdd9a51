// The grouped kinds that may cut items along the keys, bf16.
#include "prefill_kernel.cuh"

cudaError_t pkv::launch_prefill_cut_bf16(const CUtensorMap& tq, const CUtensorMap& tk,
                                      const CUtensorMap& tv, const PrefillArgs& a, int head_dim,
                                      int kind, cudaStream_t stream) {
    return head_dim == 128 ? launch_grouped<__nv_bfloat16, 128, kCut>(tq, tk, tv, a, kind, stream)
                           : launch_grouped<__nv_bfloat16, 64, kCut>(tq, tk, tv, a, kind, stream);
}
