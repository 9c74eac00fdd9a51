// Attention of new tokens over a latent cache, in the absorbed form: the cache rows
// are the keys of every head and their first R elements the values.
//
// A first version: a block a (token, head) row, a warp a token at a time, the running
// maximum and sum of the softmax per warp, the warps joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "launch.cuh"
#include "pkv_internal.h"
#include "rows16.cuh"

namespace {

using namespace pkv::rows16;

constexpr int kP = 64;

struct Args {
    uint16_t* out;
    const uint16_t *q, *cache;
    const int32_t *tables, *ctx, *q_start;
    const int64_t* ancestors;
    float scale_log2;
    int S, H, B, max_blocks, max_qlen, T;
    int64_t num_blocks;
    int32_t* err;
};

template <typename T, int R>
__global__ void __launch_bounds__(128) latent_decode_simple(const Args a) {
    pkv::pdl_wait_then_release();
    constexpr int W = R + kP, E = W / 64;   // pairs of elements a lane
    __shared__ float s_m[4], s_l[4], s_o[4][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.z, i = blockIdx.y, h = blockIdx.x;
    const int q0 = a.q_start ? a.q_start[s] : s;
    const int qlen = a.q_start ? a.q_start[s + 1] - q0 : 1, ctx = a.ctx[s];
    const bool bad = ctx < 0 || (int64_t)ctx > (int64_t)a.max_blocks * a.B || qlen < 0 ||
                     qlen > a.max_qlen || q0 < 0 || (int64_t)q0 + qlen > a.T ||
                     (ctx > 0 && qlen > ctx);
    if (bad) {
        if (threadIdx.x == 0 && i == 0 && h == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
        return;
    }
    if (i >= qlen) return;
    const int64_t row = (int64_t)(q0 + i) * a.H + h;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + row * W);
    float2 qv[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = unpack2<T>(q[32 * e + lane]);
        o[e] = make_float2(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    const int base = ctx - qlen;
    const uint64_t seen = a.ancestors ? (uint64_t)a.ancestors[q0 + i] : ~0ull;
    for (int t = warp; t < ctx; t += 4) {
        const int j = t - base;
        if (j >= 0 && (a.ancestors ? !(seen >> j & 1) : j > i)) continue;
        const int blk = a.tables[(int64_t)s * a.max_blocks + t / a.B];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) atomicOr(a.err, PKV_DEVERR_BAD_BLOCK);
            continue;
        }
        const uint32_t* k = reinterpret_cast<const uint32_t*>(
            a.cache + ((int64_t)blk * a.B + t % a.B) * W);
        float2 kv[E];
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            kv[e] = unpack2<T>(k[32 * e + lane]);
            z = fmaf(qv[e].x, kv[e].x, fmaf(qv[e].y, kv[e].y, z));
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        z *= a.scale_log2;
        const float mn = fmaxf(m, z), c = exp2f(m - mn), p = exp2f(z - mn);
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = make_float2(fmaf(o[e].x, c, p * kv[e].x), fmaf(o[e].y, c, p * kv[e].y));
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < R / 64; ++e) {
        s_o[warp][2 * (32 * e + lane)] = o[e].x;
        s_o[warp][2 * (32 * e + lane) + 1] = o[e].y;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int x = 0; x < 4; ++x) M = fmaxf(M, s_m[x]);
    for (int x = 0; x < 4; ++x) L += M == -INFINITY ? 0.f : s_l[x] * exp2f(s_m[x] - M);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * R);
    for (int d = threadIdx.x; d < R / 2; d += 128) {
        float x = 0.f, y = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
            x = fmaf(f, s_o[w][2 * d], x);
            y = fmaf(f, s_o[w][2 * d + 1], y);
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        out[d] = pack2<T>(x * inv, y * inv);
    }
}

}  // namespace

extern "C" {

pkv_status pkv_latent_decode_workspace_size(int num_seqs, int num_heads, int latent_dim,
                                            int max_query_len, size_t* bytes) {
    const char* fn = "pkv_latent_decode_workspace_size";
    if (!bytes) return pkv::fail(PKV_ERR_INVALID, "%s: bytes is NULL", fn);
    if (num_seqs < 0 || num_heads < 1 || (latent_dim != 256 && latent_dim != 512) ||
        max_query_len < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    *bytes = 256;
    return PKV_OK;
}

pkv_status pkv_latent_attention_decode(
    void* out, const void* q, const void* cache, const int32_t* block_tables,
    const int32_t* context_lens, const int32_t* query_start, const int64_t* ancestors, float scale,
    int num_seqs, int num_heads, int latent_dim, int rope_dim, int block_size,
    int max_blocks_per_seq, int64_t num_blocks, int max_query_len, int num_query_tokens,
    pkv_dtype dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    const char* fn = "pkv_latent_attention_decode";
    if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, %d]", fn, PKV_MAX_SEQS);
    if (num_heads < 1 || num_heads > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_heads must be in [1, 65535]", fn);
    if (latent_dim != 256 && latent_dim != 512)
        return pkv::fail(PKV_ERR_INVALID, "%s: latent_dim must be 256 or 512", fn);
    if (rope_dim != kP) return pkv::fail(PKV_ERR_INVALID, "%s: rope_dim must be 64", fn);
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    if (max_blocks_per_seq < 1 || max_query_len < 0 || num_query_tokens < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    if ((int64_t)max_blocks_per_seq * block_size > (1LL << 30))
        return pkv::fail(PKV_ERR_INVALID, "%s: context capacity above 2^30 tokens", fn);
    if (num_blocks < 1 || num_blocks > ((1LL << 31) - 1) / block_size)
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_blocks must be >= 1, and num_blocks * block_size below 2^31", fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    const float scale_log2 = (float)(1.4426950408889634 * scale);
    if (!std::isfinite(scale_log2))
        return pkv::fail(PKV_ERR_INVALID, "%s: scale is not finite", fn);
    if (!query_start && (num_query_tokens != num_seqs || max_query_len < 1))
        return pkv::fail(PKV_ERR_INVALID, "%s: without query_start each sequence has one row", fn);
    if (ancestors && max_query_len > 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: a tree has at most 64 rows", fn);
    if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !cache || !block_tables || !context_lens || !workspace)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(cache, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q and the cache must be 16-byte aligned", fn);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    Args a = {static_cast<uint16_t*>(out), static_cast<const uint16_t*>(q),
              static_cast<const uint16_t*>(cache), block_tables, context_lens, query_start,
              ancestors, scale_log2, num_seqs, num_heads, block_size, max_blocks_per_seq,
              max_query_len, num_query_tokens, num_blocks, err};
    using Kernel = void (*)(Args);
    const Kernel k = dtype == PKV_F16
                         ? (latent_dim == 256 ? (Kernel)latent_decode_simple<__half, 256>
                                              : (Kernel)latent_decode_simple<__half, 512>)
                         : (latent_dim == 256 ? (Kernel)latent_decode_simple<__nv_bfloat16, 256>
                                              : (Kernel)latent_decode_simple<__nv_bfloat16, 512>);
    const cudaError_t e = pkv::launch_pdl(
        k, dim3((unsigned)num_heads, (unsigned)max_query_len, (unsigned)num_seqs), dim3(128),
        stream, a);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
