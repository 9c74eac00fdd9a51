// The new tokens' way into a latent cache, and cached rows' way out of it.
//
// A latent cache holds one row a token: R elements of a latent vector, from which
// every head's key and value would be formed, then P = 64 elements of a rotated
// key part that all heads share.
//
// Write.  Per token, in fp32 and rounded once to the storage type:
//   row[0 .. R)      latent / sqrt(mean(latent^2) + eps) * w   (w given), or latent
//   row[R .. R + P)  the shared key part, turned by the token's position
//   q_out[h]         the rotary part of query head h, turned by it
// Angles are those of rope_cache.cu: fixed-point fractions of a turn, exact modulo
// one turn at any position.
//
// Bound: HBM bytes; with few tokens, latency.  A warp takes one token, or one of
// `parts` equal runs of its passes when there are few tokens: a pass is four query
// rows, 8 lanes of 8 elements a row, so that a lane owns the same four pairs of
// every row and computes their angles once; the latent row and the key part are
// one warp's, 16 or 8 latent elements a lane.
//
// Measured: 16001 tokens, 32 heads, R 256: 26.2 us (5.79 TB/s, 0.86 of a plain copy);
// 16384 tokens, 16 heads, R 512: 17.3 us (6.08 TB/s); 64 tokens 2.8 us, one 2.2.
// Passes loaded at a time: 2 took 28.2 us, 8 26.1 but 19.7 for the narrower batch; more
// blocks an SM by fewer registers 28.9; one warp a token at eight passes and more 29.9.
//
// Gather.  Rows key_start[s] + t of the output are the cached rows of tokens t of
// sequence s.  A warp moves four rows, every 16-byte piece of them loaded before
// the first is stored.  Measured: 74000 rows of R 512 26.6 us (6.44 TB/s, 0.95 of a plain
// copy; eight rows a warp 27.9), 700 rows 2.0 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "launch.cuh"
#include "pkv_internal.h"
#include "rows16.cuh"

namespace {

using namespace pkv::rows16;

constexpr int kP = 64;                      // the rotated part
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kWarpsPerSm = 12;             // aimed at when there are few tokens
constexpr int kLatentPasses = 2;            // what a token's own row counts for

struct WriteArgs {
    uint16_t* q_out;
    const uint16_t *q, *latent, *k_rope;
    int64_t qo_stride, qo_head, q_stride, q_head, latent_stride, rope_stride;   // elements
    uint16_t* cache;
    const int64_t* slots;
    const int32_t* positions;
    const uint64_t* phases;
    const float* weight;                    // null: no norm
    float eps, rope_scale;
    int T, H;
    int parts;                              // warps that share one token
    int64_t num_slots;
    int32_t* err;
};

// The four pairs that a lane turns: elements ea .. ea + 3 and eb .. eb + 3 of a row;
// pair j is element j of each or, interleaved, 2 j and 2 j + 1 of the eight.
template <bool INTERLEAVED>
struct Turn {
    uint64_t c[4], s[4];

    __device__ __forceinline__ void set(const uint64_t* phases, int li, int pos, float scale) {
        float cs[4], sn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int turn = (int)((phases[4 * li + j] * (uint64_t)(int64_t)pos) >> 32);   // 2^-32 turns
            sincospif((float)turn * 0x1p-31f, &sn[j], &cs[j]);
            cs[j] *= scale;
            sn[j] *= scale;
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
    }

    template <typename T>
    __device__ __forceinline__ void apply(uint2& a, uint2& b) const {
        const uint32_t word[4] = {a.x, a.y, b.x, b.y};
        uint64_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2<T>(word[e]);
            x[e] = two(v.x, v.y);
        }
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = split(x[e]);
                x[e] = fma2(x[e], c[e], mul2(two(v.y, v.x), s[e]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint64_t p = x[e], q = x[2 + e];
                x[e] = fma2(p, c[e], mul2(q, s[2 + e]));
                x[2 + e] = fma2(q, c[e], mul2(p, s[e]));
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = split(x[e]);
            o[e] = pack2<T>(v.x, v.y);
        }
        a = make_uint2(o[0], o[1]);
        b = make_uint2(o[2], o[3]);
    }
};

template <typename T, int R, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) latent_norm_rope_and_cache_kernel(const WriteArgs p) {
    pkv::pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = p.parts == 1 ? w : w / p.parts;
    const int part = (int)(w - t * p.parts);
    if (t >= p.T) return;
    const int li = lane & 7, sub = lane >> 3;
    const int ea = INTERLEAVED ? 8 * li : 4 * li;
    const int eb = INTERLEAVED ? ea + 4 : kP / 2 + 4 * li;
    const int nq = (p.H + 3) / 4, n = nq + kLatentPasses;
    const int i0 = p.parts == 1 ? 0 : part * n / p.parts;
    const int i1 = p.parts == 1 ? n : (part + 1) * n / p.parts;

    Turn<INTERLEAVED> turn;
    const int pos = p.positions[t];
    constexpr int L = R / 256;              // 16-byte pieces of the latent row a lane holds
    if (i0 <= nq && nq < i1) {
        const int64_t slot = p.slots[t];
        uint4 x[L];
        const uint16_t* in = p.latent + t * p.latent_stride + 8 * lane;
#pragma unroll
        for (int u = 0; u < L; ++u) x[u] = *reinterpret_cast<const uint4*>(in + 256 * u);
        uint2 ka = make_uint2(0u, 0u), kb = ka;
        if (sub == 0) {
            const uint16_t* kr = p.k_rope + t * p.rope_stride;
            ka = *reinterpret_cast<const uint2*>(kr + ea);
            kb = *reinterpret_cast<const uint2*>(kr + eb);
        }
        turn.set(p.phases, li, pos, p.rope_scale);
        turn.template apply<T>(ka, kb);
        if (p.weight) {
            float v[L][8], sum = 0.f;
#pragma unroll
            for (int u = 0; u < L; ++u) {
                const uint32_t word[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<T>(word[e]);
                    v[u][2 * e] = f.x;
                    v[u][2 * e + 1] = f.y;
                    sum = fmaf(f.x, f.x, sum);
                    sum = fmaf(f.y, f.y, sum);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = rsqrtf(sum * (1.f / R) + p.eps);
#pragma unroll
            for (int u = 0; u < L; ++u) {
                const float4* wt = reinterpret_cast<const float4*>(p.weight + 256 * u + 8 * lane);
                const float4 wa = __ldg(wt), wb = __ldg(wt + 1);
                x[u].x = pack2<T>(v[u][0] * (wa.x * r), v[u][1] * (wa.y * r));
                x[u].y = pack2<T>(v[u][2] * (wa.z * r), v[u][3] * (wa.w * r));
                x[u].z = pack2<T>(v[u][4] * (wb.x * r), v[u][5] * (wb.y * r));
                x[u].w = pack2<T>(v[u][6] * (wb.z * r), v[u][7] * (wb.w * r));
            }
        }
        if (slot >= p.num_slots && lane == 0) atomicOr(p.err, PKV_DEVERR_BAD_SLOT);
        if (slot >= 0 && slot < p.num_slots) {
            uint16_t* row = p.cache + slot * (R + kP);
#pragma unroll
            for (int u = 0; u < L; ++u) *reinterpret_cast<uint4*>(row + 256 * u + 8 * lane) = x[u];
            if (sub == 0) {
                *reinterpret_cast<uint2*>(row + R + ea) = ka;
                *reinterpret_cast<uint2*>(row + R + eb) = kb;
            }
        }
    } else {
        turn.set(p.phases, li, pos, p.rope_scale);
    }
    const uint16_t* in = p.q + t * p.q_stride;
    uint16_t* out = p.q_out + t * p.qo_stride;
    const int to = min(i1, nq), heads = min(p.H, 4 * to);
    for (int from = i0; from < to; from += kUnroll) {
        const int h0 = 4 * from + sub;
        uint2 a[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            a[u] = b[u] = make_uint2(0u, 0u);
            if (h0 + 4 * u < heads) {
                const uint16_t* row = in + (h0 + 4 * u) * p.q_head;
                a[u] = *reinterpret_cast<const uint2*>(row + ea);
                b[u] = *reinterpret_cast<const uint2*>(row + eb);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (from + u >= to) break;
            turn.template apply<T>(a[u], b[u]);
            if (h0 + 4 * u < heads) {
                uint16_t* row = out + (h0 + 4 * u) * p.qo_head;
                *reinterpret_cast<uint2*>(row + ea) = a[u];
                *reinterpret_cast<uint2*>(row + eb) = b[u];
            }
        }
    }
}

// ---------------------------------------------------------------- gather
struct GatherArgs {
    uint4* rows;
    const uint4* cache;
    const int32_t *tables, *key_start;
    int S, B, max_blocks;
    int64_t T, num_blocks;
    int32_t* err;
};

constexpr int kGatherRows = 4;

// PIECES 16-byte pieces a row
template <int PIECES>
__global__ void __launch_bounds__(kThreads) gather_latent_kernel(const GatherArgs p) {
    pkv::pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kGatherRows;
    if (r0 >= p.T) return;
    // lane i < 4 finds row r0 + i: the last sequence that begins at or before it
    int64_t from = -1;
    const int64_t row = r0 + lane;
    if (lane < kGatherRows && row < p.T) {
        int lo = 0, hi = p.S;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.key_start[mid] <= row) lo = mid;
            else hi = mid;
        }
        const int64_t t = row - p.key_start[lo];
        if (t >= 0 && row < p.key_start[lo + 1]) {
            if (t >= (int64_t)p.max_blocks * p.B) {
                atomicOr(p.err, PKV_DEVERR_BAD_CONTEXT);
            } else {
                const int64_t b = t / p.B;
                const int64_t blk = p.tables[(int64_t)lo * p.max_blocks + b];
                if (blk < 0 || blk >= p.num_blocks) atomicOr(p.err, PKV_DEVERR_BAD_BLOCK);
                else from = blk * p.B + (t - b * p.B);
            }
        }
    }
    constexpr int N = (kGatherRows * PIECES + 31) / 32;
    uint4 x[N];
    bool live[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int i = 32 * u + lane, k = i / PIECES;
        const int64_t src = __shfl_sync(0xffffffffu, from, k < kGatherRows ? k : 0);
        live[u] = k < kGatherRows && src >= 0;
        if (live[u]) x[u] = __ldcs(p.cache + src * PIECES + (i - k * PIECES));
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
        if (live[u]) p.rows[r0 * PIECES + 32 * u + lane] = x[u];
}

bool bad_sizes(const char* fn, int latent_dim, int rope_dim, int block_size, int64_t num_blocks,
               pkv_dtype dtype, pkv_status* st) {
    if (latent_dim != 256 && latent_dim != 512)
        *st = pkv::fail(PKV_ERR_INVALID, "%s: latent_dim must be 256 or 512", fn);
    else if (rope_dim != kP)
        *st = pkv::fail(PKV_ERR_INVALID, "%s: rope_dim must be 64", fn);
    else if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        *st = pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    else if (num_blocks < 1 || num_blocks > (1LL << 60) / ((latent_dim + kP) * block_size * 2))
        *st = pkv::fail(PKV_ERR_INVALID, "%s: num_blocks must be >= 1 and its pool in reach", fn);
    else if (dtype != PKV_F16 && dtype != PKV_BF16)
        *st = pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    else
        return false;
    return true;
}

template <typename T>
cudaError_t launch_write(const WriteArgs& a, int R, bool interleaved, dim3 grid,
                         cudaStream_t stream) {
    using Kernel = void (*)(WriteArgs);
    const Kernel k =
        R == 256 ? (interleaved ? (Kernel)latent_norm_rope_and_cache_kernel<T, 256, true>
                                : (Kernel)latent_norm_rope_and_cache_kernel<T, 256, false>)
                 : (interleaved ? (Kernel)latent_norm_rope_and_cache_kernel<T, 512, true>
                                : (Kernel)latent_norm_rope_and_cache_kernel<T, 512, false>);
    return pkv::launch_pdl(k, grid, dim3(kThreads), stream, a);
}

}  // namespace

extern "C" {

pkv_status pkv_latent_norm_rope_and_cache(
    void* q_out, int64_t q_out_stride, int64_t q_out_head_stride, const void* q, int64_t q_stride,
    int64_t q_head_stride, const void* latent, int64_t latent_stride, const void* k_rope,
    int64_t k_rope_stride, void* cache, const int64_t* slot_mapping, const int32_t* positions,
    const uint64_t* phases, int interleaved, float rope_scale, const float* weight, float eps,
    int num_tokens, int num_heads, int latent_dim, int rope_dim, int block_size,
    int64_t num_blocks, pkv_dtype dtype, cudaStream_t stream) {
    const char* fn = "pkv_latent_norm_rope_and_cache";
    pkv_status st;
    if (bad_sizes(fn, latent_dim, rope_dim, block_size, num_blocks, dtype, &st)) return st;
    if (num_heads < 1 || num_heads > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_heads must be in [1, 65535]", fn);
    if (!std::isfinite(rope_scale))
        return pkv::fail(PKV_ERR_INVALID, "%s: rope_scale is not finite", fn);
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return pkv::fail(PKV_ERR_INVALID, "%s: eps must be finite and not negative", fn);
    if (num_tokens < 0 || num_tokens > (1 << 28))
        return pkv::fail(PKV_ERR_INVALID, "%s: num_tokens must be in [0, 2^28]", fn);
    const int64_t most = 1LL << 32;
    const int64_t strides[6] = {q_out_stride, q_out_head_stride, q_stride, q_head_stride,
                                latent_stride, k_rope_stride};
    for (int64_t s : strides)
        if (s < kP || s % 8 != 0 || s > most)
            return pkv::fail(PKV_ERR_INVALID,
                             "%s: strides must cover a row, be multiples of 8 elements and at "
                             "most 2^32",
                             fn);
    const int64_t qo_span = (num_heads - 1) * q_out_head_stride + kP;
    const int64_t q_span = (num_heads - 1) * q_head_stride + kP;
    if (q_out_stride < qo_span || q_stride < q_span || latent_stride < latent_dim)
        return pkv::fail(PKV_ERR_INVALID, "%s: token strides must cover a token's rows", fn);
    if (num_tokens == 0) return PKV_OK;
    if (!q_out || !q || !latent || !k_rope || !cache || !slot_mapping || !positions || !phases)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(latent, 16) || !aligned(k_rope, 16) ||
        !aligned(cache, 16) || !aligned(weight, 16))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: q_out, q, latent, k_rope, the cache and the weight must be 16-byte "
                         "aligned",
                         fn);
    if (!aligned(slot_mapping, 8) || !aligned(phases, 8) || !aligned(positions, 4))
        return pkv::fail(PKV_ERR_INVALID, "%s: misaligned slot_mapping, phases or positions", fn);
    // different warps read and write the rows: q_out may be q itself, row for row, and
    // must otherwise share nothing with the inputs
    const int64_t nt = num_tokens - 1;
    const int64_t out_bytes = (nt * q_out_stride + qo_span) * 2;
    const bool in_place =
        q_out == q && q_stride == q_out_stride && q_head_stride == q_out_head_stride;
    const struct {
        const void* at;
        int64_t bytes;
    } in[3] = {{q, (nt * q_stride + q_span) * 2},
               {latent, (nt * latent_stride + latent_dim) * 2},
               {k_rope, (nt * k_rope_stride + kP) * 2}};
    const int64_t pool_bytes = num_blocks * block_size * (latent_dim + kP) * 2;
    for (int i = 0; i < 3; ++i) {
        if (!(i == 0 && in_place) && overlap(q_out, out_bytes, in[i].at, in[i].bytes))
            return pkv::fail(PKV_ERR_INVALID, "%s: q_out overlaps an input", fn);
        if (overlap(cache, pool_bytes, in[i].at, in[i].bytes))
            return pkv::fail(PKV_ERR_INVALID, "%s: the cache overlaps an input", fn);
    }
    if (overlap(cache, pool_bytes, q_out, out_bytes))
        return pkv::fail(PKV_ERR_INVALID, "%s: the cache overlaps q_out", fn);

    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    const int sms = pkv::sm_count(dev);
    if (sms < 1) return pkv::fail(PKV_ERR_CUDA, "%s: no multiprocessors", fn);

    WriteArgs a;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q = static_cast<const uint16_t*>(q);
    a.latent = static_cast<const uint16_t*>(latent);
    a.k_rope = static_cast<const uint16_t*>(k_rope);
    a.qo_stride = q_out_stride;
    a.qo_head = q_out_head_stride;
    a.q_stride = q_stride;
    a.q_head = q_head_stride;
    a.latent_stride = latent_stride;
    a.rope_stride = k_rope_stride;
    a.cache = static_cast<uint16_t*>(cache);
    a.slots = slot_mapping;
    a.positions = positions;
    a.phases = phases;
    a.weight = weight;
    a.eps = eps;
    a.rope_scale = rope_scale;
    a.T = num_tokens;
    a.H = num_heads;
    a.num_slots = num_blocks * block_size;
    a.err = err;
    // warps per token: enough that every SM has about kWarpsPerSm of them, at most one
    // per pass
    const int64_t passes = (num_heads + 3) / 4 + kLatentPasses;
    const int64_t parts = ((int64_t)sms * kWarpsPerSm + num_tokens - 1) / num_tokens;
    a.parts = (int)(parts < passes ? parts : passes);
    const int64_t warps = (int64_t)num_tokens * a.parts;
    const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
    e = dtype == PKV_F16 ? launch_write<__half>(a, latent_dim, interleaved != 0, grid, stream)
                         : launch_write<__nv_bfloat16>(a, latent_dim, interleaved != 0, grid,
                                                       stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

pkv_status pkv_gather_latent(void* rows, const void* cache, const int32_t* block_tables,
                             const int32_t* key_start, int num_seqs, int latent_dim, int rope_dim,
                             int block_size, int max_blocks_per_seq, int64_t num_blocks,
                             int num_rows, pkv_dtype dtype, cudaStream_t stream) {
    const char* fn = "pkv_gather_latent";
    pkv_status st;
    if (bad_sizes(fn, latent_dim, rope_dim, block_size, num_blocks, dtype, &st)) return st;
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, 65535]", fn);
    if (max_blocks_per_seq < 1 || num_rows < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    if (num_seqs == 0 || num_rows == 0) return PKV_OK;
    if (!rows || !cache || !block_tables || !key_start)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(rows, 16) || !aligned(cache, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: rows and the cache must be 16-byte aligned", fn);
    if (!aligned(block_tables, 4) || !aligned(key_start, 4))
        return pkv::fail(PKV_ERR_INVALID, "%s: misaligned block_tables or key_start", fn);
    const int64_t row_bytes = (latent_dim + kP) * 2;
    if (overlap(rows, num_rows * row_bytes, cache, num_blocks * block_size * row_bytes))
        return pkv::fail(PKV_ERR_INVALID, "%s: rows overlaps the cache", fn);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    GatherArgs a;
    a.rows = static_cast<uint4*>(rows);
    a.cache = static_cast<const uint4*>(cache);
    a.tables = block_tables;
    a.key_start = key_start;
    a.S = num_seqs;
    a.B = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.T = num_rows;
    a.num_blocks = num_blocks;
    a.err = err;
    const int64_t warps = ((int64_t)num_rows + kGatherRows - 1) / kGatherRows;
    const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
    using Kernel = void (*)(GatherArgs);
    const Kernel k = latent_dim == 256 ? (Kernel)gather_latent_kernel<(256 + kP) / 8>
                                       : (Kernel)gather_latent_kernel<(512 + kP) / 8>;
    const cudaError_t e = pkv::launch_pdl(k, grid, dim3(kThreads), stream, a);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
