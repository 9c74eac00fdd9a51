// C ABI of the prompt phase: argument checks, tensor maps and launch of the
// plain kernel (prefill_kernel.cuh), with or without the cache write.
#include "prefill_kernel.cuh"

namespace {

pkv_status prefill_common(const char* fn, void* out, const void* q, const void* k_in,
                          const void* v_in, void* k_cache, void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens,
                          const int32_t* query_start, float scale, int num_seqs, int num_heads,
                          int head_dim, int block_size, int max_blocks_per_seq,
                          int64_t num_blocks, int max_query_len, int num_query_tokens,
                          pkv_dtype dtype, cudaStream_t stream) {
    const bool fused = k_in != nullptr || v_in != nullptr;
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, 65535]", fn);
    if (num_heads < 1 || num_heads > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_heads must be in [1, 65535]", fn);
    if (head_dim != 64 && head_dim != 128)
        return pkv::fail(PKV_ERR_INVALID, "%s: head_dim must be 64 or 128", fn);
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    if (max_blocks_per_seq < 1 || num_blocks < 1 || max_query_len < 0 || num_query_tokens < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    if ((int64_t)max_blocks_per_seq * block_size >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: context capacity overflows", fn);
    // the tiled copies address cache rows (block, head, token) with 32-bit coordinates
    if (num_blocks * num_heads * block_size >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: pool too large for 32-bit row coordinates", fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16) return pkv::fail(PKV_ERR_INVALID, "%s: dtype", fn);
    {
        // the work schedule sums item costs in 64 bits: a bound far above any
        // call whose tensors fit in memory
        const double units = (double)((num_heads + 1) / 2) * num_seqs *
                             (double)(((int64_t)max_query_len + kRows - 1) / kRows);
        const double unit_cost =
            kPairCost * ((double)max_blocks_per_seq * block_size / kBN + 1.0) + kItemCost;
        if (units * unit_cost >= 0x1p60)
            return pkv::fail(PKV_ERR_INVALID, "%s: too much work for one call", fn);
    }
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f)
        return pkv::fail(PKV_ERR_INVALID, "%s: scale is not finite", fn);
    if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start ||
        (fused && (!k_in || !v_in)))
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        (fused && (!aligned(k_in, 16) || !aligned(v_in, 16))))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q, k, v and the caches must be 16-byte aligned",
                         fn);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);

    const bool bf16 = dtype == PKV_BF16;
    const cuuint64_t D = (cuuint64_t)head_dim;
    CUtensorMap tq, tk, tv, tkin, tvin;
    {
        // q (and the prompt's k, v): [tokens][heads][D], one box = 128 tokens
        // x 64 elements of one head
        const cuuint64_t dims[3] = {D, (cuuint64_t)num_heads, (cuuint64_t)num_query_tokens};
        const cuuint64_t strides[2] = {D * 2, (cuuint64_t)num_heads * D * 2};
        const cuuint32_t box[3] = {64, 1, (cuuint32_t)kBM};
        if (!make_map(&tq, bf16, 3, q, dims, strides, box))
            return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of q", fn);
        if (fused) {
            if (!make_map(&tkin, bf16, 3, k_in, dims, strides, box) ||
                !make_map(&tvin, bf16, 3, v_in, dims, strides, box))
                return pkv::fail(PKV_ERR_CUDA, "%s: tensor maps of k and v", fn);
        } else {
            tkin = tq;                       // unused
            tvin = tq;
        }
    }
    {
        // caches: rows (block, head, token) of D elements, one box = one block's
        // tokens x 64 elements
        const cuuint64_t dims[2] = {D, (cuuint64_t)(num_blocks * num_heads * block_size)};
        const cuuint64_t strides[1] = {D * 2};
        const cuuint32_t box[2] = {64, (cuuint32_t)block_size};
        if (!make_map(&tk, bf16, 2, k_cache, dims, strides, box) ||
            !make_map(&tv, bf16, 2, v_cache, dims, strides, box))
            return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of the caches", fn);
    }
    PrefillArgs a = {};
    a.out = out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.out_v8 = aligned(out, 32) ? 1 : 0;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.S = num_seqs;
    a.H = num_heads;
    a.B = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.max_query_len = max_query_len;
    a.num_tokens = num_query_tokens;
    a.q_items = (max_query_len + kRows - 1) / kRows;
    a.num_blocks = num_blocks;
    a.err = err;
    cudaError_t e;
    if (fused) {
        if (!bf16)
            e = head_dim == 128
                    ? launch_prefill<__half, 128, true, kPlain>(tq, tk, tv, tkin, tvin, a, stream)
                    : launch_prefill<__half, 64, true, kPlain>(tq, tk, tv, tkin, tvin, a, stream);
        else
            e = head_dim == 128
                    ? launch_prefill<__nv_bfloat16, 128, true, kPlain>(tq, tk, tv, tkin, tvin, a, stream)
                    : launch_prefill<__nv_bfloat16, 64, true, kPlain>(tq, tk, tv, tkin, tvin, a, stream);
    } else {
        if (!bf16)
            e = head_dim == 128
                    ? launch_prefill<__half, 128, false, kPlain>(tq, tk, tv, tkin, tvin, a, stream)
                    : launch_prefill<__half, 64, false, kPlain>(tq, tk, tv, tkin, tvin, a, stream);
        else
            e = head_dim == 128
                    ? launch_prefill<__nv_bfloat16, 128, false, kPlain>(tq, tk, tv, tkin, tvin, a, stream)
                    : launch_prefill<__nv_bfloat16, 64, false, kPlain>(tq, tk, tv, tkin, tvin, a, stream);
    }
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_paged_attention_prefill(void* out, const void* q, const void* k_cache,
                                       const void* v_cache, const int32_t* block_tables,
                                       const int32_t* context_lens, const int32_t* query_start,
                                       float scale, int num_seqs, int num_heads, int head_dim,
                                       int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                       int max_query_len, int num_query_tokens, pkv_dtype dtype,
                                       cudaStream_t stream) {
    return prefill_common("pkv_paged_attention_prefill", out, q, nullptr, nullptr,
                          const_cast<void*>(k_cache), const_cast<void*>(v_cache), block_tables,
                          context_lens, query_start, scale, num_seqs, num_heads, head_dim,
                          block_size, max_blocks_per_seq, num_blocks, max_query_len,
                          num_query_tokens, dtype, stream);
}

pkv_status pkv_paged_attention_prefill_write(void* out, const void* q, const void* k,
                                             const void* v, void* k_cache, void* v_cache,
                                             const int32_t* block_tables,
                                             const int32_t* context_lens,
                                             const int32_t* query_start, float scale,
                                             int num_seqs, int num_heads, int head_dim,
                                             int block_size, int max_blocks_per_seq,
                                             int64_t num_blocks, int max_query_len,
                                             int num_query_tokens, pkv_dtype dtype,
                                             cudaStream_t stream) {
    const char* fn = "pkv_paged_attention_prefill_write";
    if (!k || !v) return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    return prefill_common(fn, out, q, k, v, k_cache, v_cache, block_tables, context_lens,
                          query_start, scale, num_seqs, num_heads, head_dim, block_size,
                          max_blocks_per_seq, num_blocks, max_query_len, num_query_tokens, dtype,
                          stream);
}

}  // extern "C"
