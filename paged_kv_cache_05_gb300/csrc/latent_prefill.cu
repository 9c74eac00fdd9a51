// Attention of prompts in the expanded form of latent attention: a head's keys are N
// elements of its own and 64 that all heads share, its values N elements.
//
// A first version: a block a (token, head) row, a warp a key at a time, the running
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
    const uint16_t *q, *k, *k_rope, *v;
    int64_t q_stride, q_head, k_stride, k_head, r_stride, v_stride, v_head;
    const int32_t *q_start, *k_start;
    float scale_log2;
    int S, H, max_q, max_k, Tq, Tk;
    int32_t* err;
};

template <typename T, int N>
__global__ void __launch_bounds__(128) latent_prefill_simple(const Args a) {
    pkv::pdl_wait_then_release();
    constexpr int E = (N + kP) / 64, V = N / 64;
    __shared__ float s_m[4], s_l[4], s_o[4][N];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.z, h = blockIdx.y, i = blockIdx.x;
    const int q0 = a.q_start[s], k0 = a.k_start[s];
    const int qlen = a.q_start[s + 1] - q0, klen = a.k_start[s + 1] - k0;
    if (qlen < 0 || qlen > a.max_q || q0 < 0 || (int64_t)q0 + qlen > a.Tq || klen < qlen ||
        klen > a.max_k || k0 < 0 || (int64_t)k0 + klen > a.Tk) {
        if (threadIdx.x == 0 && i == 0 && h == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
        return;
    }
    if (i >= qlen) return;
    const int64_t row = q0 + i;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + row * a.q_stride + h * a.q_head);
    float2 qv[E], o[V];
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = unpack2<T>(q[32 * e + lane]);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    const int end = klen - qlen + i + 1;
    for (int t = warp; t < end; t += 4) {
        const int64_t at = k0 + t;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k + at * a.k_stride + h * a.k_head);
        const uint32_t* r = reinterpret_cast<const uint32_t*>(a.k_rope + at * a.r_stride);
        const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + at * a.v_stride + h * a.v_head);
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 x = unpack2<T>(e < V ? k[32 * e + lane] : r[lane]);
            z = fmaf(qv[e].x, x.x, fmaf(qv[e].y, x.y, z));
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        z *= a.scale_log2;
        const float mn = fmaxf(m, z), c = exp2f(m - mn), p = exp2f(z - mn);
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 x = unpack2<T>(v[32 * e + lane]);
            o[e] = make_float2(fmaf(o[e].x, c, p * x.x), fmaf(o[e].y, c, p * x.y));
        }
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_o[warp][2 * (32 * e + lane)] = o[e].x;
        s_o[warp][2 * (32 * e + lane) + 1] = o[e].y;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int x = 0; x < 4; ++x) M = fmaxf(M, s_m[x]);
    for (int x = 0; x < 4; ++x) L += M == -INFINITY ? 0.f : s_l[x] * exp2f(s_m[x] - M);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (row * a.H + h) * N);
    for (int d = threadIdx.x; d < N / 2; d += 128) {
        float x = 0.f, y = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
            x = fmaf(f, s_o[w][2 * d], x);
            y = fmaf(f, s_o[w][2 * d + 1], y);
        }
        out[d] = pack2<T>(x / L, y / L);
    }
}

}  // namespace

extern "C" {

pkv_status pkv_latent_attention_prefill(
    void* out, const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
    int64_t k_stride, int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
    const void* v, int64_t v_stride, int64_t v_head_stride, const int32_t* query_start,
    const int32_t* key_start, float scale, int num_seqs, int num_heads, int head_dim, int rope_dim,
    int max_query_len, int max_key_len, int num_query_tokens, int num_key_tokens, pkv_dtype dtype,
    cudaStream_t stream) {
    const char* fn = "pkv_latent_attention_prefill";
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, 65535]", fn);
    if (num_heads < 1 || num_heads > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_heads must be in [1, 65535]", fn);
    if (head_dim != 64 && head_dim != 128)
        return pkv::fail(PKV_ERR_INVALID, "%s: head_dim must be 64 or 128", fn);
    if (rope_dim != kP) return pkv::fail(PKV_ERR_INVALID, "%s: rope_dim must be 64", fn);
    if (max_query_len < 0 || max_key_len < 0 || num_query_tokens < 0 || num_key_tokens < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    const float scale_log2 = (float)(1.4426950408889634 * scale);
    if (!std::isfinite(scale_log2))
        return pkv::fail(PKV_ERR_INVALID, "%s: scale is not finite", fn);
    const struct {
        int64_t token, head, row;
        const char* name;
    } st[4] = {{q_stride, q_head_stride, head_dim + kP, "q"},
               {k_stride, k_head_stride, head_dim, "k"},
               {k_rope_stride, kP, kP, "k_rope"},
               {v_stride, v_head_stride, head_dim, "v"}};
    for (const auto& x : st)
        if (x.token < x.row || x.head < x.row || x.token % 8 != 0 || x.head % 8 != 0 ||
            x.token > (1LL << 32) || x.head > (1LL << 32))
            return pkv::fail(PKV_ERR_INVALID,
                             "%s: strides of %s must cover a row, be multiples of 8 elements and "
                             "at most 2^32",
                             fn, x.name);
    if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !query_start || !key_start || !k || !k_rope || !v)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(k_rope, 16) ||
        !aligned(v, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q, k, k_rope and v must be 16-byte aligned",
                         fn);
    if (!aligned(query_start, 4) || !aligned(key_start, 4))
        return pkv::fail(PKV_ERR_INVALID, "%s: misaligned query_start or key_start", fn);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    Args a = {static_cast<uint16_t*>(out), static_cast<const uint16_t*>(q),
              static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(k_rope),
              static_cast<const uint16_t*>(v), q_stride, q_head_stride, k_stride, k_head_stride,
              k_rope_stride, v_stride, v_head_stride, query_start, key_start, scale_log2, num_seqs,
              num_heads, max_query_len, max_key_len, num_query_tokens, num_key_tokens, err};
    using Kernel = void (*)(Args);
    const Kernel kernel =
        dtype == PKV_F16 ? (head_dim == 64 ? (Kernel)latent_prefill_simple<__half, 64>
                                           : (Kernel)latent_prefill_simple<__half, 128>)
                         : (head_dim == 64 ? (Kernel)latent_prefill_simple<__nv_bfloat16, 64>
                                           : (Kernel)latent_prefill_simple<__nv_bfloat16, 128>);
    const cudaError_t e = pkv::launch_pdl(
        kernel, dim3((unsigned)max_query_len, (unsigned)num_heads, (unsigned)num_seqs), dim3(128),
        stream, a);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
