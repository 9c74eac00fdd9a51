// The new tokens' way into the cache: norm of queries and keys per head,
// rotation by position, and the write of K and V into their slots, in one
// pass over the projections' output.
//
// Per head row x[0 .. D) of a query or key (fp32 arithmetic, one rounding to
// the storage type at the end):
//   norm      x <- x / sqrt(mean(x^2) + eps) * w          (optional, per kind)
//   rotation  the pair (a, b) of index i turns by angle = position * f_i:
//             (a, b) <- rope_scale * (a cos - b sin, b cos + a sin)
// where pair i is (x[i], x[i + rot/2]) or, interleaved, (x[2i], x[2i + 1]),
// and elements from rot on are left alone.  Values are copied bit for bit.
//
// Angles.  position * f_i in fp32 is off by radians at far positions, so
// frequencies come as 64-bit binary fractions of a turn (units of 2^-64
// turns): the product position * phase modulo 2^64 is the exact angle modulo
// one turn in one integer multiplication.  Its upper 32 bits, as a signed
// number, go through sincospif (|angle| at most half a turn, error 2^-24 of
// it), so no table of cosines is kept or read.
//
// Bound: HBM bytes (each row read once, written once), with instruction issue
// close behind (a first version at 170 instructions a pass was bound by it, at
// 5.3 TB/s): hence one walk per kind of row, weights in registers, packed fp32
// pairs.  Layout of the work: a warp takes one token, or one of `parts` equal
// runs of its rows when there are few tokens; D/8 lanes hold a row (8 elements
// each, so that a lane owns the same four pairs of every row it meets and
// computes their angles once), 2 or 4 rows fill the warp (a pass), and kUnroll
// passes are loaded before the first is computed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "launch.cuh"
#include "pkv_internal.h"
#include "rows16.cuh"

namespace {

using namespace pkv::rows16;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
// Resident blocks per SM that the registers are allotted for (73 a thread):
// 16384 tokens of 32 + 8 + 8 heads of 128 take 63.1 us (6.38 TB/s), against 67.3
// for 6 and 67.4 for 9.
constexpr int kResident = 7;
constexpr int kWarpsPerSm = 12;             // aimed at when there are few tokens
constexpr int kLongToken = 16;              // passes of a token that is given two warps

struct RopeArgs {
    uint16_t* q_out;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    uint16_t *k_cache, *v_cache;
    const int64_t* slots;
    const int32_t* positions;
    const uint64_t* phases;
    const float *q_weight, *k_weight;       // null: no norm
    float eps, rope_scale;
    int T, H, HK, rot, B;
    int parts;                              // warps that share one token
    int64_t num_slots;
    int32_t* err;
};

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kResident) norm_rope_and_cache_kernel(const RopeArgs p) {
    pkv::pdl_wait_then_release();
    constexpr int LPR = D / 8;              // lanes per row
    constexpr int RPP = 32 / LPR;           // rows per pass
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = p.parts == 1 ? w : w / p.parts;
    const int part = (int)(w - t * p.parts);
    if (t >= p.T) return;
    // a lane holds four elements of a row at offset ea and four at eb; where its
    // pairs turn, pair j is element j of each (interleaved: 2 j and 2 j + 1 of
    // the eight, which are consecutive)
    const int li = lane % LPR, sub = lane / LPR;
    const bool turns = li < p.rot / 8;
    const int ea = INTERLEAVED ? 8 * li : turns ? 4 * li : 8 * li;
    const int eb = INTERLEAVED || !turns ? ea + 4 : p.rot / 2 + 4 * li;

    // passes of the token: its query rows, key rows, value rows; this warp takes
    // an equal run of them, kUnroll loaded at a time
    const int nq = (p.H + RPP - 1) / RPP, nk = (p.HK + RPP - 1) / RPP, n = nq + 2 * nk;
    const int i0 = p.parts == 1 ? 0 : part * n / p.parts;
    const int i1 = p.parts == 1 ? n : (part + 1) * n / p.parts;
    const int64_t slot = p.slots[t];
    const int pos = p.positions[t];
    uint64_t c[4], s[4];
    bool ready = false;
    auto angles = [&]() {
        ready = true;
        if (!turns) return;
        float cs[4], sn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int turn = (int)((p.phases[4 * li + j] * (uint64_t)(int64_t)pos) >> 32);   // 2^-32 turns
            sincospif((float)turn * 0x1p-31f, &sn[j], &cs[j]);
            cs[j] *= p.rope_scale;
            sn[j] *= p.rope_scale;
        }
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = two(cs[j], cs[j]);
                s[j] = two(-sn[j], sn[j]);
            }
        } else {
            c[0] = two(cs[0], cs[1]);
            c[1] = two(cs[2], cs[3]);
            s[0] = two(sn[0], sn[1]);
            s[1] = two(sn[2], sn[3]);
            s[2] = two(-sn[0], -sn[1]);
            s[3] = two(-sn[2], -sn[3]);
        }
    };

    // passes [from, to) of one kind: head h at src + h * D, its result at dst + h * dst_head
    auto rows = [&](const uint16_t* src, uint16_t* dst, int64_t dst_head, int heads, int from,
                    int to, const float* wt) {
        uint64_t wv[4];
        if (wt) {
            const float4 wa = __ldg(reinterpret_cast<const float4*>(wt + ea));
            const float4 wb = __ldg(reinterpret_cast<const float4*>(wt + eb));
            wv[0] = two(wa.x, wa.y);
            wv[1] = two(wa.z, wa.w);
            wv[2] = two(wb.x, wb.y);
            wv[3] = two(wb.z, wb.w);
        }
        heads = min(heads, to * RPP);
        for (; from < to; from += kUnroll) {
            uint2 xa[kUnroll], xb[kUnroll];
            const int h0 = from * RPP + sub;
            const uint16_t* in = src + h0 * D;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                xa[u] = xb[u] = make_uint2(0u, 0u);
                if (h0 + u * RPP < heads) {
                    xa[u] = *reinterpret_cast<const uint2*>(in + u * RPP * D + ea);
                    xb[u] = *reinterpret_cast<const uint2*>(in + u * RPP * D + eb);
                }
            }
            if (!ready) angles();
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (from + u >= to) break;
                const int h = h0 + u * RPP;
                const uint32_t word[4] = {xa[u].x, xa[u].y, xb[u].x, xb[u].y};
                uint64_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = unpack2<T>(word[e]);
                    x[e] = two(v.x, v.y);
                }
                if (wt) {
                    uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) sq = fma2(x[e], x[e], sq);
                    const float2 v = split(sq);
                    float sum = v.x + v.y;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float r = rsqrtf(sum * (1.f / D) + p.eps);
                    const uint64_t r2 = two(r, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], mul2(wv[e], r2));
                }
                if (turns) {
                    if constexpr (INTERLEAVED) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = split(x[e]);
                            x[e] = fma2(x[e], c[e], mul2(two(v.y, v.x), s[e]));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint64_t a = x[e], b = x[2 + e];
                            x[e] = fma2(a, c[e], mul2(b, s[2 + e]));
                            x[2 + e] = fma2(b, c[e], mul2(a, s[e]));
                        }
                    }
                }
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = split(x[e]);
                    o[e] = pack2<T>(v.x, v.y);
                }
                if (h < heads) {
                    uint16_t* to = dst + h * dst_head;
                    *reinterpret_cast<uint2*>(to + ea) = make_uint2(o[0], o[1]);
                    *reinterpret_cast<uint2*>(to + eb) = make_uint2(o[2], o[3]);
                }
            }
        }
    };
    rows(p.q + t * p.q_stride, p.q_out + t * p.H * D, D, p.H, i0, min(i1, nq), p.q_weight);
    if (slot >= p.num_slots && part == 0 && lane == 0) atomicOr(p.err, PKV_DEVERR_BAD_SLOT);
    if (slot < 0 || slot >= p.num_slots) return;
    const int64_t blk = slot / p.B;
    const int64_t at = (blk * p.HK * p.B + slot - blk * p.B) * D, head = (int64_t)p.B * D;
    rows(p.k + t * p.k_stride, p.k_cache + at, head, p.HK, max(i0 - nq, 0), min(i1 - nq, nk),
         p.k_weight);
    // values, as they are
    const int to = min(i1 - nq - nk, nk), heads = min(p.HK, to * RPP);
    for (int from = max(i0 - nq - nk, 0); from < to; from += kUnroll) {
        const int h0 = from * RPP + sub;
        const uint16_t* in = p.v + t * p.v_stride + h0 * D + 8 * li;
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h0 + u * RPP < heads) x[u] = *reinterpret_cast<const uint4*>(in + u * RPP * D);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h0 + u * RPP < heads)
                *reinterpret_cast<uint4*>(p.v_cache + at + (h0 + u * RPP) * head + 8 * li) = x[u];
    }
}

template <typename T>
cudaError_t launch(const RopeArgs& a, int D, bool interleaved, dim3 grid, cudaStream_t stream) {
    using Kernel = void (*)(RopeArgs);
    const Kernel k = D == 64 ? (interleaved ? (Kernel)norm_rope_and_cache_kernel<T, 64, true>
                                            : (Kernel)norm_rope_and_cache_kernel<T, 64, false>)
                             : (interleaved ? (Kernel)norm_rope_and_cache_kernel<T, 128, true>
                                            : (Kernel)norm_rope_and_cache_kernel<T, 128, false>);
    return pkv::launch_pdl(k, grid, dim3(kThreads), stream, a);
}

}  // namespace

extern "C" {

pkv_status pkv_rope_inv_freq(int rot_dim, double base, pkv_rope_scaling scaling, double factor,
                             int original_len, double beta_fast, double beta_slow,
                             double* inv_freq, float* rope_scale) {
    const char* fn = "pkv_rope_inv_freq";
    if (!inv_freq || !rope_scale) return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 4096)
        return pkv::fail(PKV_ERR_INVALID, "%s: rot_dim must be even, in [2, 4096]", fn);
    if (!(base > 1.0) || !std::isfinite(base))
        return pkv::fail(PKV_ERR_INVALID, "%s: base must be above 1", fn);
    if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_BY_PARTS)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown scaling", fn);
    if (scaling != PKV_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return pkv::fail(PKV_ERR_INVALID, "%s: factor must be at least 1", fn);
    if (scaling == PKV_ROPE_BASE && rot_dim == 2)
        return pkv::fail(PKV_ERR_INVALID, "%s: a larger base needs rot_dim above 2", fn);
    double low = 0.0, high = 0.0;
    if (scaling == PKV_ROPE_BY_PARTS) {
        if (original_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
            !std::isfinite(beta_fast))
            return pkv::fail(PKV_ERR_INVALID,
                             "%s: scaling by parts needs original_len >= 1 and "
                             "0 < beta_slow < beta_fast",
                             fn);
        // YaRN (Peng, Quesnelle, Fan, Shippole, 2023): a ramp between the pairs that
        // make beta_fast and beta_slow turns over the original length, its ends on
        // whole pairs, never empty, and attention scaled by 0.1 ln(factor) + 1.
        // The (fractional) pair that makes `turns` turns:
        auto pair_of = [&](double turns) {
            return rot_dim * std::log(original_len / (turns * 6.283185307179586)) /
                   (2.0 * std::log(base));
        };
        low = std::floor(pair_of(beta_fast));
        high = std::ceil(pair_of(beta_slow));
        if (low < 0.0) low = 0.0;
        if (high > rot_dim - 1) high = rot_dim - 1;
        if (!(high > low)) high = low + 0.001;
    }
    if (scaling == PKV_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    *rope_scale = 1.f;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == PKV_ROPE_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_BY_PARTS) {
            double slow = (i - low) / (high - low);      // 0: kept, 1: slowed by factor
            slow = slow < 0.0 ? 0.0 : slow > 1.0 ? 1.0 : slow;
            f = f / factor * slow + f * (1.0 - slow);
        }
        inv_freq[i] = f;
    }
    if (scaling == PKV_ROPE_BY_PARTS) *rope_scale = (float)(0.1 * std::log(factor) + 1.0);
    return PKV_OK;
}

pkv_status pkv_rope_phases(const double* inv_freq, int n, uint64_t* phases) {
    const char* fn = "pkv_rope_phases";
    if (n < 0) return pkv::fail(PKV_ERR_INVALID, "%s: n < 0", fn);
    if (n > 0 && (!inv_freq || !phases)) return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(inv_freq[i]))
            return pkv::fail(PKV_ERR_INVALID, "%s: frequency %d is not finite", fn, i);
    for (int i = 0; i < n; ++i) {
        const double turns = inv_freq[i] / 6.283185307179586;
        const double part = turns - std::floor(turns);   // [0, 1], 1 only by rounding
        phases[i] = part < 1.0 ? (uint64_t)std::ldexp(part, 64) : 0;
    }
    return PKV_OK;
}

pkv_status pkv_norm_rope_and_cache(void* q_out, const void* q, const void* k, const void* v,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                   const int32_t* positions, const uint64_t* phases, int rot_dim,
                                   int interleaved, float rope_scale, const float* q_weight,
                                   const float* k_weight, float eps, int num_tokens,
                                   int num_heads, int num_kv_heads, int head_dim, int block_size,
                                   int64_t num_blocks, pkv_dtype dtype, cudaStream_t stream) {
    const char* fn = "pkv_norm_rope_and_cache";
    if (num_heads < 1 || num_kv_heads < 1 || num_heads > 65535 || num_kv_heads > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: head counts must be in [1, 65535]", fn);
    if (head_dim != 64 && head_dim != 128)
        return pkv::fail(PKV_ERR_INVALID, "%s: head_dim must be 64 or 128", fn);
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    if (num_blocks < 1 ||
        num_blocks > (1LL << 60) / ((int64_t)num_kv_heads * head_dim * block_size * 2))
        return pkv::fail(PKV_ERR_INVALID, "%s: num_blocks must be >= 1 and its pool in reach", fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 8 != 0)
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: rot_dim must be a multiple of 8 in [0, head_dim]", fn);
    if (!std::isfinite(rope_scale))
        return pkv::fail(PKV_ERR_INVALID, "%s: rope_scale is not finite", fn);
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return pkv::fail(PKV_ERR_INVALID, "%s: eps must be finite and not negative", fn);
    if (num_tokens < 0 || num_tokens > (1 << 28))
        return pkv::fail(PKV_ERR_INVALID, "%s: num_tokens must be in [0, 2^28]", fn);
    const int64_t qd = (int64_t)num_heads * head_dim, kd = (int64_t)num_kv_heads * head_dim;
    if (q_stride < qd || k_stride < kd || v_stride < kd || q_stride % 8 != 0 ||
        k_stride % 8 != 0 || v_stride % 8 != 0 || q_stride > (1LL << 32) ||
        k_stride > (1LL << 32) || v_stride > (1LL << 32))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: token strides must cover the heads, be multiples of 8 elements and "
                         "at most 2^32",
                         fn);
    if (num_tokens == 0) return PKV_OK;
    if (!q_out || !q || !k || !v || !k_cache || !v_cache || !slot_mapping || !positions ||
        (rot_dim > 0 && !phases))
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: q_out, q, k, v, the caches and the weights must be 16-byte aligned",
                         fn);
    if (!aligned(slot_mapping, 8) || !aligned(phases, 8) || !aligned(positions, 4))
        return pkv::fail(PKV_ERR_INVALID, "%s: misaligned slot_mapping, phases or positions", fn);
    // rows are read and written by different warps: q_out may be q itself, row
    // for row, and must otherwise share nothing with the inputs
    const int64_t nt = num_tokens - 1;
    const int64_t out_bytes = (nt + 1) * qd * 2;
    const bool in_place = q_out == q && q_stride == qd;
    if ((!in_place && overlap(q_out, out_bytes, q, (nt * q_stride + qd) * 2)) ||
        overlap(q_out, out_bytes, k, (nt * k_stride + kd) * 2) ||
        overlap(q_out, out_bytes, v, (nt * v_stride + kd) * 2))
        return pkv::fail(PKV_ERR_INVALID, "%s: q_out overlaps an input", fn);
    const int64_t pool_bytes = num_blocks * block_size * kd * 2;
    const void* pools[2] = {k_cache, v_cache};
    for (const void* pool : pools)
        if (overlap(pool, pool_bytes, q_out, out_bytes) ||
            overlap(pool, pool_bytes, q, (nt * q_stride + qd) * 2) ||
            overlap(pool, pool_bytes, k, (nt * k_stride + kd) * 2) ||
            overlap(pool, pool_bytes, v, (nt * v_stride + kd) * 2))
            return pkv::fail(PKV_ERR_INVALID, "%s: a cache overlaps an input or q_out", fn);
    if (overlap(k_cache, pool_bytes, v_cache, pool_bytes))
        return pkv::fail(PKV_ERR_INVALID, "%s: the caches overlap", fn);

    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    const int sms = pkv::sm_count(dev);
    if (sms < 1) return pkv::fail(PKV_ERR_CUDA, "%s: no multiprocessors", fn);

    RopeArgs a;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_cache = static_cast<uint16_t*>(k_cache);
    a.v_cache = static_cast<uint16_t*>(v_cache);
    a.slots = slot_mapping;
    a.positions = positions;
    a.phases = phases;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.rope_scale = rope_scale;
    a.T = num_tokens;
    a.H = num_heads;
    a.HK = num_kv_heads;
    a.rot = rot_dim;
    a.B = block_size;
    a.num_slots = num_blocks * block_size;
    a.err = err;
    // Warps per token: enough that every SM has about kWarpsPerSm of them, two for
    // long tokens while all stay resident (2000 tokens of 40 + 8 + 8 heads of 128:
    // 14.7 -> 12.5 us), at most one per pass of rows.
    const int rpp = 256 / head_dim;
    const int64_t passes = (num_heads + rpp - 1) / rpp + 2 * ((num_kv_heads + rpp - 1) / rpp);
    int64_t parts = ((int64_t)sms * kWarpsPerSm + num_tokens - 1) / num_tokens;
    if (parts == 1 && passes >= kLongToken &&
        2 * (int64_t)num_tokens <= (int64_t)sms * kResident * kWarps)
        parts = 2;
    a.parts = (int)(parts < passes ? parts : passes);
    const int64_t warps = (int64_t)num_tokens * a.parts;
    const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
    e = dtype == PKV_F16 ? launch<__half>(a, head_dim, interleaved != 0, grid, stream)
                         : launch<__nv_bfloat16>(a, head_dim, interleaved != 0, grid, stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
