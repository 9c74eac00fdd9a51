// Attention of new tokens over a latent cache, in the absorbed form: the cache rows
// (W = R + 64 elements) are the keys of every head and their first R elements the
// values.  Per (token, head) row, over the tokens t it sees:
//   z_t = scale q . row_t,   out = sum_t 2^(z_t - m) row_t[0 .. R) / sum_t 2^(z_t - m)
// in log2 units, with the running max and sum of the softmax (one pass over the cache).
//
// Every head of a token attends the same rows, so a tile is 128 (token, head) rows of
// one sequence, 128 cached tokens a step, and both products are matrix products:
// 2 x 128 x 128 x (W + R) operations on 128 x 2 W bytes, at 128 heads 242 a byte, near
// the 284 at which the tensor cores and the memory take the same time.  An output of
// 128 x 512 in fp32 is all of an SM's tensor memory, and 128 query rows and a tile of
// tokens exceed its shared memory, so a tile is a pair of CTAs' (cluster of two, one
// product by both, cta_group::2):
//   S = Q K^T      each CTA holds 64 query rows (A) and 64 of the tile's tokens (half
//                  of B's columns), and gets 64 x 128 scores in 64 columns: lanes 0-63
//                  its rows against tokens 0-63, lanes 64-127 against tokens 64-127
//   O += P V       each CTA holds its rows' weights P (A) and half of the values' R
//                  elements of all 128 tokens (half of B's columns)
// R = 256 takes half of that, so that a pair can hold a tile of 256 rows as well, 128 a CTA:
// a lane a row, its scores in 128 columns, weights over the scores.
// A token's row thus comes to each CTA of the pair in part as a key and in part as a
// value, 17/9 of its bytes in all: the copies' rate into the SMs (10-11 TB/s of boxes
// of 8 rows, measured) bounds long contexts at 5.8 TB/s of the cache.  A step of R = 512 is
// 36 products for S (N = 128, 50 cycles each, measured back to back) and 16 for O (N = 256,
// 64): 2800 cycles of the 5000 that a step of 128 heads takes; what the rest is has not been
// measured.
//
// Measured (graph of calls, the joining kernel counted): 8 sequences of 8192-32768, 16
// heads, R 512: 49.8 us (4.0 TB/s of the cache); 64 of 1-2048, 128 heads, R 512: 39.0 us;
// 33 trees of 13 behind 77-4095, 20 heads, R 256: 31.2 us; one sequence of 500, 16 heads:
// 9.9 us.  Boxes of 16 and more rows free a step's keys later (53 us for the long ones),
// one thread issuing a step's boxes in turn 57, prefetches into L2 changed nothing.
//
// Eight warps a CTA (256 rows: twelve):
//   warp 0      keys: boxes of 8 rows x KC chunks of 64 elements, one lane a box (lanes'
//               copies start side by side, a thread's one after the other), a ring of
//               KS slots of KC chunks of the tile's 64 tokens, freed slot by slot as S
//               is formed
//   warp 6      values: boxes of 8 rows x R / 128 chunks, a ring of VS slots of 32 tokens
//   warp 7      queries
//   warp 1      (of the first CTA) issues the products
//   warps 2-5   softmax (256 rows: 8-11 too): a thread a row and half of the tile's tokens;
//               the two halves of a row meet in shared memory.  The max is raised only
//               past a growth of kRescale, so that most steps leave O alone.
// S is double-buffered: S of step j + 1 is formed while the softmax of step j runs.
//
// The steps of all (sequence, row tile)s are dealt to the pairs in equal runs.  A run
// that holds all steps of one writes its output rows; parts of one are left in the
// workspace (fp32 output, max and sum), and a second kernel joins them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_internal.h"
#include "rows16.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace {

using namespace pkv::tc;
using pkv::rows16::aligned;
using pkv::rows16::overlap;
using pkv::rows16::pack2;

constexpr int kP = 64;
constexpr int kTok = 128;             // tokens of a step
constexpr int kMaxPairs = 96;

template <int R, int TILE>
struct Cfg {
    static constexpr int W = R + kP;
    static constexpr int CH = W / 64;                 // chunks of a row
    static constexpr int VCH = R / 128;               // chunks of a CTA's half of the values
    static constexpr int KC = R == 512 ? 3 : 5;       // chunks of a key slot
    static constexpr int KSUB = CH / KC;              // slots of a step
    static constexpr int KS = R == 512 ? 3 : 2;
    static constexpr int VS = R == 512 ? 4 : TILE == 128 ? 8 : 7;
    static constexpr bool WIDE = TILE == 256;         // P over S in tensor memory
    static constexpr int RC = TILE / 2;               // rows of a CTA
    static constexpr int SOFTMAX = RC / 16;           // its softmax warps
    static constexpr int WARPS = 4 + SOFTMAX;
    static constexpr int THREADS = 32 * WARPS;
    // tensor memory: two of S, then O
    static constexpr uint32_t COL_S = RC;             // columns of one
    static constexpr uint32_t COL_O = 2 * COL_S;
    static constexpr int K_SLOT = KC * 8192;
    static constexpr int V_GROUP = VCH * 1024;        // 8 tokens
    static constexpr int V_SLOT = 4 * V_GROUP;
    static constexpr int Q_BYTES = CH * RC * 128;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + Q_BYTES;
    static constexpr int V_OFF = K_OFF + KS * K_SLOT;
    static constexpr int P_OFF = V_OFF + VS * V_SLOT;
    static constexpr int P_BYTES = WIDE ? 0 : 16384;
    static constexpr int SMEM = P_OFF + P_BYTES + 1024;   // 1 KiB of alignment slack
    static_assert(SMEM + (WIDE ? 3072 : 2048) <= 232448, "shared memory");
    static_assert(COL_O + R * TILE / 256 <= 512, "tensor memory");
    static_assert(KSUB * KC == CH, "chunks");
};

enum : int {
    kKFull = 0,      // + slot (up to 3): both CTAs' keys are there (first CTA's barrier)
    kKEmpty = 3,     // + slot
    kVFull = 6,      // + slot (up to 8)
    kVEmpty = 14,    // + slot
    kSFull = 22,     // + buffer
    kPFull = 24,     // weights written by all softmax warps (first CTA's)
    kPvDone = 25,    // O += P V of a step completed
    kQFull = 26,
    kQEmpty = 27,    // a segment's last S formed
    kORead = 28,     // a segment's output read from tensor memory (first CTA's)
    kBars = 29
};

struct Args {
    uint16_t* out;
    const uint16_t* cache;
    const int32_t *tables, *ctx, *q_start;
    const int64_t* ancestors;
    float scale_log2;
    int S, H, B, max_blocks, max_qlen, T;
    int64_t num_blocks;
    int pairs, slot_rows;             // rows of a part in the workspace
    int log_rows;                     // of a tile
    int out_v8;                       // out is 32-byte aligned: 32-byte stores
    struct Rec* rec;                  // [pairs]
    float2* ml;                       // [2 pairs][slot_rows]
    float* acc;                       // [2 pairs][R / 8][slot_rows][8]
    int32_t* err;
    uint64_t wait_ns;                 // of a wait (pkv_set_decode_wait_limit)
};

// What is left to join: rows of the output whose parts lie in `parts` slots: `slot`,
// then the first of each following pair.
struct Rec {
    int row0, rows, slot, parts;
};

struct Seq {
    int q0, qlen, ctx;
    int nt, nr;                       // steps of a row tile, row tiles (0: nothing to do)
    // what a sequence's lengths are, as they lie in memory ...
    __device__ __forceinline__ void fetch(const Args& a, int s) {
        q0 = a.q_start ? a.q_start[s] : s;
        qlen = a.q_start ? a.q_start[s + 1] : s + 1;
        ctx = a.ctx[s];
    }
    // ... and looked at (the loads are waited for here)
    __device__ __forceinline__ bool look(const Args& a) {
        qlen -= q0;
        nt = nr = 0;
        if (ctx < 0 || (int64_t)ctx > (int64_t)a.max_blocks * a.B || qlen < 0 ||
            qlen > a.max_qlen || q0 < 0 || (int64_t)q0 + qlen > a.T || (ctx > 0 && qlen > ctx))
            return false;
        if (qlen > 0 && ctx > 0) {
            nt = (ctx + kTok - 1) / kTok;
            nr = (int)(((int64_t)qlen * a.H + (1 << a.log_rows) - 1) >> a.log_rows);
        }
        return true;
    }
    __device__ __forceinline__ bool load(const Args& a, int s) {
        fetch(a, s);
        return look(a);
    }
    __device__ __forceinline__ int64_t steps() const { return (int64_t)nt * nr; }
};

// Where a pair's run begins.
struct Start {
    int s;
    Seq q;
    int64_t off, n;                   // steps before it in the sequence, steps of the run
    int64_t total;                    // steps of all
};

// A run of steps of one row tile.
struct Seg {
    int s, q0, qlen, ctx;
    int row;                          // first row of the tile among the sequence's
    int rows;                         // live rows of the tile
    int j0, j1;                       // steps
    bool whole;
    int slot;                         // of a part: 0 the run's first, 1 another
};

struct Walker {
    Seq q, next;
    int s;
    int64_t off, left;
    bool first;
    __device__ __forceinline__ void init(const Args& a, const Start& st) {
        s = st.s;
        off = st.off;
        left = st.n;
        first = true;
        q = st.q;
        if (left > 0 && s + 1 < a.S) next.fetch(a, s + 1);
    }
    __device__ __forceinline__ bool get(const Args& a, Seg& g) {
        if (left <= 0) return false;
        while (off >= q.steps()) {
            if (++s >= a.S) return false;
            off = 0;
            q = next;
            q.look(a);
            if (s + 1 < a.S) next.fetch(a, s + 1);
        }
        const int rt = off < (1 << 30) ? (int)off / q.nt : (int)(off / q.nt);
        g.s = s;
        g.q0 = q.q0;
        g.qlen = q.qlen;
        g.ctx = q.ctx;
        g.row = rt << a.log_rows;
        g.rows = min(1 << a.log_rows, q.qlen * a.H - g.row);
        g.j0 = (int)(off - (int64_t)rt * q.nt);
        g.j1 = (int)min((int64_t)q.nt, g.j0 + left);
        g.whole = g.j0 == 0 && g.j1 == q.nt;
        g.slot = first ? 0 : 1;
        first = false;
        off += g.j1 - g.j0;
        left -= g.j1 - g.j0;
        return true;
    }
};

// The block of a sequence's token and the cache row of it, or -1.
__device__ __forceinline__ int cache_row(const Args& a, const Seg& g, int t) {
    if (t >= g.ctx) return -1;
    const int b = t / a.B;
    const int id = a.tables[(int64_t)g.s * a.max_blocks + b];
    if (id < 0 || id >= a.num_blocks) return -1;
    return id * a.B + (t - b * a.B);
}

// The values of a step that holds drafted tokens of a tree that no row attends, whose places may
// hold anything: groups with such places are copied by the warp, zeros in those (a weight of 0
// does not hide a value that is not finite), the others as ever.  Lane i < 16: group i's row y and
// which of its 8 tokens to keep; `none`: a row past the pool; vc: slots filled so far.  Returns
// vc after the step or, if a wait ran out, ~vc as it is by then.  (Not inlined: within the warp's
// loop it cost calls without trees 2 %.)
template <class C>
__device__ __noinline__ int fill_kept(const uint16_t* cache, const CUtensorMap* map, uint32_t bar0,
                                      uint32_t values, int none, int subs, int y, uint32_t keep, int vc,
                                      const volatile Limit* limit) {
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    if (keep == 0) y = -1;
    const uint32_t parts = __ballot_sync(0xffffffffu, lane < 16 && keep != 0 && keep != 0xffu);
    for (int v = 0; v < subs; ++v, ++vc) {
        const int st = vc % C::VS, n = vc / C::VS;
        if (n > 0 && !warp_wait(bar0 + 8 * (kVEmpty + st), (uint32_t)((n - 1) & 1), limit)) return ~vc;
        const uint32_t full = at_rank(bar0 + 8 * (kVFull + st), 0);
        const uint32_t slot = values + st * C::V_SLOT;
        const uint32_t which = parts >> 4 * v & 15u;
        for (uint32_t rest = which; rest; rest &= rest - 1) {
            const int at = __ffs(rest) - 1;
            const int yt = __shfl_sync(0xffffffffu, y, 4 * v + at);
            const uint32_t kept = __shfl_sync(0xffffffffu, keep, 4 * v + at);
            for (int i = lane; i < C::VCH * 64; i += 32) {
                const int r = i / (C::VCH * 8), c = i - r * (C::VCH * 8);
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (yt >= 0 && (kept >> r & 1))
                    w = *reinterpret_cast<const uint4*>(cache + (int64_t)(yt + r) * C::W +
                                                        rank * ((C::W - kP) / 2) + c * 8);
                st_shared_v4(slot + at * C::V_GROUP + (c >> 3) * 1024 + r * 128 + (((c & 7) ^ r) << 4),
                             w.x, w.y, w.z, w.w);
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_expect_tx_cluster(full, (4 - __popc(which)) * C::V_GROUP);
        __syncwarp();
        if ((lane >> 2) == v && !(parts >> lane & 1))
            tma_3d_pair(slot + (lane & 3) * C::V_GROUP, map, 0, y < 0 ? none : y, rank * C::VCH, full);
    }
    return vc;
}

// Either CTA gave up: what is in flight ends before they do, products (by their commits, of
// which the first CTA keeps count) and copies (counted by roles that gave up; one that did
// not has seen the last of its ring used).  bar0: the barriers, used0: the phases used of each
// ring, at its first barrier's place.  (Not inlined, and no count kept otherwise: those cost
// calls that never come here up to 3 %.)
template <class C>
__device__ __noinline__ void end_given_up(uint32_t bar0, uint32_t used0) {
    cluster_sync();
    if (threadIdx.x < 32) {
        const uint32_t rank = cluster_rank();
        volatile Limit longest = {kWaitLimitNs, 0};     // (whatever the call's)
        auto used = [&](int b, uint32_t r) { return ld_cluster(at_rank(used0 + 4 * b, r)); };
        auto products = [&](int b, int slots) { ring_ended(bar0 + 8 * b, slots, used(b, 0), &longest); };
        auto copies = [&](int b, int slots) {
            if (rank == 0) copies_ended(bar0 + 8 * b, slots, used(b, 0), used(b, 1));
        };
        products(kKEmpty, C::KS);
        products(kVEmpty, C::VS);
        products(kSFull, 2);
        products(kPvDone, 1);
        products(kQEmpty, 1);
        copies(kKFull, C::KS);
        copies(kVFull, C::VS);
        copies(kQFull, 1);
    }
    fence_before();
    __syncthreads();
    cluster_sync();
}

// Tokens of a group of 8, by bits: those before the sequence's end, `n` tokens on ...
__device__ __forceinline__ uint32_t kept_of(int n) { return n >= 8 ? 0xffu : n > 0 ? (1u << n) - 1 : 0u; }
// ... and of them those that are not drafted or that some row of the tree attends (`bits`, each
// lane those of some rows).  One warp.
__device__ __noinline__ uint32_t attended(uint64_t bits, int qlen, int n) {
    const uint64_t gone = ~((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32)) << 32 |
                            __reduce_or_sync(0xffffffffu, (uint32_t)bits));
    const int d = qlen - n;                          // the group's first, drafted
    return kept_of(n) & ~(d >= 64 || d <= -8 ? 0u : d >= 0 ? (uint32_t)(gone >> d) : (uint32_t)(gone << -d));
}

template <typename T, int R, int TILE>
__global__ void __launch_bounds__(Cfg<R, TILE>::THREADS, 1)
    latent_decode_pair(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using C = Cfg<R, TILE>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ uint32_t s_tmem;
    __shared__ Limit s_limit;
    __shared__ int s_used[kBars];                   // phases of a ring, at its first barrier's place
    __shared__ Start s_start;
    __shared__ int64_t s_scan[2][C::WARPS];
    __shared__ float s_x[2][2][C::RC];              // a row's maxima (or sums) by halves

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = (int)(blockIdx.x >> 1);
    volatile Limit* const limit = &s_limit;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sQ = base + C::Q_OFF, sK = base + C::K_OFF, sV = base + C::V_OFF,
                   sP = base + C::P_OFF;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the pair's run of the steps: [b, e) of all (the lengths are loaded once where
    // there is a thread a sequence, and on their way while the barriers are made)
    Seq mine;
    mine.nt = mine.nr = 0;
    bool good = tid >= a.S || mine.load(a, tid);
    if (warp == 1) {
        for (int i = lane; i < kBars; i += 32) {
            const bool two = i < kKEmpty || (i >= kVFull && i < kVEmpty) || i == kQFull;
            mbar_init(bar(i), two ? 2 : i == kPFull || i == kORead ? 2 * C::SOFTMAX : 1);
        }
        mbar_init_fence();
        for (int i = lane; i < kBars; i += 32) s_used[i] = kNotCounted;
        if (lane == 0) s_limit = Limit{a.wait_ns, 0};
        __syncwarp();
        alloc_pair(smem_u32(&s_tmem));
    } else if (warp == 0 && lane == 0) {
        prefetch_map(&tm_q);
        prefetch_map(&tm_k);
        prefetch_map(&tm_v);
    }
    {
        // this thread's steps, and those of the threads before it in the warp
        int64_t n = mine.steps(), incl = n, rest = 0;
        for (int s = tid + C::THREADS; s < a.S; s += C::THREADS) {
            Seq q;
            good &= q.load(a, s);
            rest += q.steps();
        }
        if (!good && blockIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (a.S > C::THREADS) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
        }
        if (lane == 31) {
            s_scan[0][warp] = incl;
            s_scan[1][warp] = rest;
        }
        if (tid == 0) s_start.n = 0;
        fence_before();
        __syncthreads();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // (see mbar_init_fence)
        int64_t total = 0, before = 0;
        for (int w = 0; w < C::WARPS; ++w) {
            if (w < warp) incl += s_scan[0][w];
            before += s_scan[0][w];
            total += s_scan[0][w] + s_scan[1][w];
        }
        const int64_t np = min((int64_t)a.pairs, total);
        const int64_t b = pair < np ? run_begin(total, np, pair) : 0;
        const int64_t e = pair < np ? run_begin(total, np, pair + 1) : 0;
        auto found = [&](int s) {                // the sequence that holds step b
            if (e > b && incl > b && incl - n <= b) s_start = Start{s, mine, b - (incl - n), e - b, total};
        };
        found(tid);
        for (int s0 = C::THREADS; s0 < a.S && before <= b && e > b; s0 += C::THREADS) {
            mine.nt = mine.nr = 0;
            if (s0 + tid < a.S) mine.load(a, s0 + tid);
            n = incl = mine.steps();
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) s_scan[0][warp] = incl;
            __syncthreads();
            incl += before;
            for (int w = 0; w < C::WARPS; ++w) {
                if (w < warp) incl += s_scan[0][w];
                before += s_scan[0][w];
            }
            found(s0 + tid);
        }
        // (nothing to join, until a part is left)
        if (tid == 0 && rank == 0) a.rec[pair] = Rec{0, 0, 0, 0};
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    fence_after();
    const uint32_t tmem = s_tmem;
    const Start start = s_start;
    bool ok = true;
    auto fail = [&]() {
        if (!limit->gave_up) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        limit->gave_up = 1;
        set_cluster(at_rank(smem_u32(&s_limit.gave_up), cluster_rank() ^ 1), 1);
    };

    if (warp == 0) {
        // ================================================= keys
        Walker wk;
        wk.init(a, start);
        Seg g;
        int kc = 0;
        const int none = (int)min(a.num_blocks * a.B, (int64_t)0x7fffffff);   // past the pool: zeros
        while (ok && wk.get(a, g)) {
            auto row_of = [&](int j) {
                return lane < 8 ? cache_row(a, g, j * kTok + 64 * (int)rank + 8 * lane) : -1;
            };
            int y = row_of(g.j0);
            for (int j = g.j0; j < g.j1; ++j) {
                const int yn = j + 1 < g.j1 ? row_of(j + 1) : -1;
#pragma unroll
                for (int u = 0; u < C::KSUB; ++u, ++kc) {
                    const int st = kc % C::KS, n = kc / C::KS;
                    if (n > 0 && !warp_wait(bar(kKEmpty + st), (uint32_t)((n - 1) & 1), limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = at_rank(bar(kKFull + st), 0);
                    if (lane == 0) mbar_expect_tx_relaxed(full, C::K_SLOT);
                    __syncwarp();
                    if (lane < 8)
                        tma_3d_pair(sK + st * C::K_SLOT + lane * C::KC * 1024, &tm_k, 0,
                                    y < 0 ? none : y, u * C::KC, full);
                }
                if (!ok) break;
                y = yn;
            }
        }
        // (the products' last releases arrive before the CTA ends: see cluster_meet)
        ok = ok && ring_ended(bar(kKEmpty), C::KS, kc, limit);
        if (!ok) {
            if (lane == 0) s_used[kKFull] = kc;
            fail();
        }
    } else if (warp == 7) {
        // ================================================= queries
        Walker wk;
        wk.init(a, start);
        Seg g;
        const uint32_t qfull = at_rank(bar(kQFull), 0);
        int segs = 0;
        for (; wk.get(a, g); ++segs) {
            if (segs > 0 && !warp_wait(bar(kQEmpty), (uint32_t)((segs - 1) & 1), limit)) {
                ok = false;
                break;
            }
            const bool live = g.rows > C::RC * (int)rank;
            if (lane == 0) mbar_expect_tx_relaxed(qfull, live ? C::Q_BYTES : 0);
            __syncwarp();
            if (live && lane < C::RC / 8)
                tma_3d_pair(sQ + lane * C::CH * 1024, &tm_q, 0,
                            g.q0 * a.H + g.row + C::RC * (int)rank + 8 * lane, 0, qfull);
        }
        ok = ok && ring_ended(bar(kQEmpty), 1, segs, limit);
        if (!ok) {
            if (lane == 0) s_used[kQFull] = segs;
            fail();
        }
    } else if (warp == 6) {
        // ================================================= values
        Walker wk;
        wk.init(a, start);
        Seg g;
        int vc = 0;
        const int none = (int)min(a.num_blocks * a.B, (int64_t)0x7fffffff);
        while (ok && wk.get(a, g)) {
            auto row_of = [&](int j) {
                return lane < 16 ? cache_row(a, g, j * kTok + 8 * lane) : -1;
            };
            int y = row_of(g.j0);
            uint64_t bits[2] = {0, 0};                       // of the lane's rows of a tree
            if (a.ancestors) {
                if (lane < g.qlen) bits[0] = (uint64_t)a.ancestors[g.q0 + lane];
                if (lane + 32 < g.qlen) bits[1] = (uint64_t)a.ancestors[g.q0 + lane + 32];
            }
            for (int j = g.j0; j < g.j1; ++j) {
                const int yn = j + 1 < g.j1 ? row_of(j + 1) : -1;
                const int left = g.ctx - j * kTok;           // tokens of the step and after
                const int subs = left >= kTok ? 4 : (left + 31) / 32;
                // a block past the pool is left out
                if (lane < 16 && y < 0 && 8 * lane < left && rank == 0)
                    atomicOr(a.err, PKV_DEVERR_BAD_BLOCK);
                if (a.ancestors && left < g.qlen + kTok) {
                    const uint32_t keep = attended(bits[0] | bits[1], g.qlen, left - 8 * lane);
                    if (__any_sync(0xffffffffu, lane < 16 && keep != kept_of(left - 8 * lane))) {
                        vc = fill_kept<C>(a.cache, &tm_v, bar(0), sV, none, subs, y, keep, vc, limit);
                        if (vc < 0) {
                            vc = ~vc;
                            ok = false;
                            break;
                        }
                        y = yn;
                        continue;
                    }
                }
                // the group that holds the last token and places behind it, whose
                // values may be anything: copied by the warp, zeros behind the last
                const int tail = left < kTok && (left & 7) ? left >> 3 : -1;
                for (int v = 0; v < subs; ++v, ++vc) {
                    const int st = vc % C::VS, n = vc / C::VS;
                    if (n > 0 && !warp_wait(bar(kVEmpty + st), (uint32_t)((n - 1) & 1), limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = at_rank(bar(kVFull + st), 0);
                    const uint32_t slot = sV + st * C::V_SLOT;
                    const bool has_tail = (tail >> 2) == v;
                    if (has_tail) {
                        const int yt = __shfl_sync(0xffffffffu, y, tail & 15);
                        const uint32_t to = slot + (tail & 3) * C::V_GROUP;
                        uint4 w[2 * C::VCH];
#pragma unroll
                        for (int e = 0; e < 2 * C::VCH; ++e) {
                            const int i = 32 * e + lane, r = i / (C::VCH * 8), c = i - r * (C::VCH * 8);
                            w[e] = make_uint4(0u, 0u, 0u, 0u);
                            if (yt >= 0 && r < (left & 7))
                                w[e] = *reinterpret_cast<const uint4*>(
                                    a.cache + (int64_t)(yt + r) * C::W + (int)rank * (R / 2) + c * 8);
                        }
#pragma unroll
                        for (int e = 0; e < 2 * C::VCH; ++e) {
                            const int i = 32 * e + lane, r = i / (C::VCH * 8), c = i - r * (C::VCH * 8);
                            st_shared_v4(to + (c >> 3) * 1024 + r * 128 + (((c & 7) ^ r) << 4), w[e].x,
                                         w[e].y, w[e].z, w[e].w);
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        if (has_tail) mbar_expect_tx_cluster(full, 3 * C::V_GROUP);
                        else mbar_expect_tx_relaxed(full, C::V_SLOT);
                    }
                    __syncwarp();
                    if ((lane >> 2) == v && lane != tail)
                        tma_3d_pair(slot + (lane & 3) * C::V_GROUP, &tm_v, 0, y < 0 ? none : y,
                                    (int)rank * C::VCH, full);
                }
                if (!ok) break;
                y = yn;
            }
        }
        ok = ok && ring_ended(bar(kVEmpty), C::VS, vc, limit);
        if (!ok) {
            if (lane == 0) s_used[kVFull] = vc;
            fail();
        }
    } else if (warp == 1) {
        // ================================================= products
        if (rank == 0 && elect_one()) {
            constexpr uint32_t ID_S = idesc(El<T>::kType, false, kTok, TILE);
            constexpr uint32_t ID_PV = idesc(El<T>::kType, true, 256, TILE);
            const uint64_t dQ = sdesc(sQ, 16, C::CH * 1024), dK = sdesc(sK, 16, C::KC * 1024),
                           dV = sdesc(sV, 1024, C::V_GROUP), dP = sdesc(sP, 16, 1024);
            Walker wk;
            wk.init(a, start);
            Seg g;
            int kc = 0, vc = 0, sc = 0, pc = 0, qc = 0, segs = 0;
            auto k_full = [&](int k) { return bar(kKFull + k % C::KS); };
            auto k_par = [&](int k) { return (uint32_t)((k / C::KS) & 1); };
            auto v_full = [&](int v) { return bar(kVFull + v % C::VS); };
            auto v_par = [&](int v) { return (uint32_t)((v / C::VS) & 1); };
            bool have = wk.get(a, g);
            while (ok && have) {
                const Seg cur = g;
                have = wk.get(a, g);
                auto pv = [&](int j) {
                    if (!mbar_wait<false>(bar(kPFull), (uint32_t)(pc & 1), limit)) return false;
                    if (j == cur.j0 && segs > 0 &&
                        !mbar_wait<false>(bar(kORead), (uint32_t)((segs - 1) & 1), limit))
                        return false;
                    const int left = cur.ctx - j * kTok;
                    const int subs = left >= kTok ? 4 : (left + 31) / 32;
                    // (unrolled: a jump back costs the issuing thread 200 cycles)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        if (v >= subs) break;
                        if (!mbar_wait<false>(v_full(vc), v_par(vc), limit)) return false;
                        fence_after();
                        const uint64_t da = dP + (uint64_t)(((v >> 1) * 8192 + (v & 1) * 64) >> 4);
                        const uint64_t db = dV + (uint64_t)(((vc % C::VS) * C::V_SLOT) >> 4);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
#pragma unroll
                            for (int n = 0; n < R / 256; ++n) {
                                const uint64_t b = db + ((k * 2 * C::V_GROUP + n * 2048) >> 4);
                                const bool add = j > cur.j0 || v > 0 || k > 0;
                                if (!C::WIDE)
                                    umma_pair(tmem + C::COL_O + n * 128, da + 2 * k, b, ID_PV, add);
                                else
                                    umma_ts_pair(tmem + C::COL_O,
                                                 tmem + (pc & 1) * C::COL_S + (2 * v + k) * 8, b,
                                                 ID_PV, add);
                            }
                        }
                        commit_pair(bar(kVEmpty + vc % C::VS));
                        ++vc;
                    }
                    commit_pair(bar(kPvDone));
                    ++pc;
                    return true;
                };
                if (!mbar_wait<false>(bar(kQFull), (uint32_t)(segs & 1), limit)) {
                    ok = false;
                    break;
                }
                for (int j = cur.j0; ok && j < cur.j1; ++j) {
                    // the weights that these scores overwrite have been read
                    if (C::WIDE && pc > 0 &&
                        !mbar_wait<false>(bar(kPvDone), (uint32_t)((pc - 1) & 1), limit)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int u = 0; u < C::KSUB; ++u, ++kc) {
                        if (!mbar_wait<false>(k_full(kc), k_par(kc), limit)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint64_t da = dQ + (uint64_t)((u * C::KC * 1024) >> 4);
                        const uint64_t db = dK + (uint64_t)(((kc % C::KS) * C::K_SLOT) >> 4);
#pragma unroll
                        for (int i = 0; i < C::KC * 4; ++i) {
                            const int c = i >> 2, k = i & 3;
                            umma_pair(tmem + (sc & 1) * C::COL_S, da + ((c * 1024 + k * 32) >> 4),
                                      db + ((c * 1024 + k * 32) >> 4), ID_S, u > 0 || i > 0);
                        }
                        commit_pair(bar(kKEmpty + kc % C::KS));
                    }
                    if (!ok) break;
                    commit_pair(bar(kSFull + (sc & 1)));
                    ++sc;
                    if (j == cur.j1 - 1) {
                        commit_pair(bar(kQEmpty));
                        ++qc;
                    }
                    if (j > cur.j0 && !pv(j - 1)) ok = false;
                }
                if (ok && !pv(cur.j1 - 1)) ok = false;
                ++segs;
            }
            // the last output's readers, of both CTAs, have arrived before this one ends
            if (ok && segs > 0)
                ok = mbar_wait<false>(bar(kORead), (uint32_t)((segs - 1) & 1), limit);
            s_used[kKEmpty] = kc;
            s_used[kVEmpty] = vc;
            s_used[kSFull] = sc;
            s_used[kPvDone] = pc;
            s_used[kQEmpty] = qc;
            if (!ok) fail();
        }
        __syncwarp();
    } else {
        // ================================================= softmax
        // its block of 32 rows, its half of the tile's tokens: those of lanes 64-127 of a
        // product of 128 rows, of the columns' second half of one of 256
        const int quad = warp & 3, half = C::WIDE ? warp >> 3 : quad >> 1;
        const int block = C::WIDE ? quad : quad & 1;
        const int rl = block * 32 + lane;                    // row of this CTA's
        const uint32_t scol = C::WIDE ? half * 64 : 0, ocol = C::WIDE ? half * (R / 2) : 0;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t pfull = at_rank(bar(kPFull), 0), oread = at_rank(bar(kORead), 0);
        // sequences without a token: rows of zero
        for (int s = pair * 2 + (int)rank; warp < 6 && s < a.S; s += 2 * a.pairs) {
            Seq q;
            if (!q.load(a, s) || q.ctx != 0 || q.qlen == 0) continue;
            uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)q.q0 * a.H * R);
            const int64_t n = (int64_t)q.qlen * a.H * R / 8;
            for (int64_t i = tid - 64; i < n; i += 128) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        Walker wk;
        wk.init(a, start);
        Seg g;
        int sc = 0, par = 0;
        const uint64_t scale2 = f2(a.scale_log2, a.scale_log2);
        while (wk.get(a, g)) {
            const int row = C::RC * (int)rank + rl;          // of the tile
            const bool live = C::RC * (int)rank + block * 32 < g.rows;   // the warp's
            const int i = (g.row + min(row, g.rows - 1)) / a.H;            // its token
            const int first = g.ctx - g.qlen;                // tokens that every row sees
            // the new tokens that the row sees, by bits (a chain's row i: the first i + 1)
            uint64_t bits = 0;
            int sees = first + i + 1;
            if (a.ancestors) {
                sees = first;
                bits = (uint64_t)a.ancestors[g.q0 + i];
                if (g.qlen < 64) bits &= (1ull << g.qlen) - 1;
            }
            // the row's weights are 2^(z - m), its scores z at most m + kLift + kRescale:
            // m is the largest so far, or a little less, lowered by the lift
            float m = -INFINITY;
            uint64_t l2 = 0;                                 // two partial sums
            for (int j = g.j0; j < g.j1; ++j, ++sc) {
                const int t0 = j * kTok + 64 * half;         // the thread's first token
                const int t_group = t0 + 8 * (lane & 7);
                // groups of 8 tokens whose block is in the pool
                uint32_t groups = 0xffu;
                if (live) {
                    const bool in = t_group >= g.ctx || cache_row(a, g, t_group) >= 0;
                    groups = __ballot_sync(0xffffffffu, in) & 0xffu;
                }
                ok = ok && warp_wait(bar(kSFull + (sc & 1)), (uint32_t)((sc >> 1) & 1), limit);
                fence_after();
                uint32_t w[32];
                float alpha = 1.f;
                if (live) {
                    uint32_t z[64];
                    ld64(tmem + lanes + (uint32_t)(sc & 1) * C::COL_S + scol, z);
                    ld_wait(z);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x, y;
                        f2_split(mul2(f2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])),
                                      scale2),
                                 x, y);
                        z[2 * e] = __float_as_uint(x);
                        z[2 * e + 1] = __float_as_uint(y);
                    }
                    if (t0 + 64 > first || groups != 0xffu) {
                        const int n = sees - t0;             // tokens seen without bits
                        uint64_t see = n >= 64 ? ~0ull : n > 0 ? (1ull << n) - 1 : 0ull;
                        if (bits) see |= n >= 64 ? 0ull : n >= 0 ? bits << n : n > -64 ? bits >> -n : 0ull;
                        uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
                        if (groups != 0xffu) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (!(groups >> k & 1)) lo &= ~(0xffu << 8 * k);
                                if (!(groups >> (k + 4) & 1)) hi &= ~(0xffu << 8 * k);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (!((e < 32 ? lo >> e : hi >> (e - 32)) & 1))
                                z[e] = __float_as_uint(-INFINITY);
                    }
                    float top = __uint_as_float(z[0]);
#pragma unroll
                    for (int e = 1; e < 63; e += 2)
                        top = max3(top, __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
                    top = fmaxf(top, __uint_as_float(z[63]));
                    s_x[par][half][rl] = top;
                    named_sync(1 + block, 64);
                    top = fmaxf(top, s_x[par][1 - half][rl]);
                    par ^= 1;
                    if (top - m > El<T>::kLift + El<T>::kRescale && top > -INFINITY) {
                        // (rounded up: with scores so large that they are further apart
                        // than the lift, m is the largest itself, and its weight 1)
                        const float mn = __fadd_ru(top, -El<T>::kLift);
                        alpha = ex2(m - mn);
                        m = mn;
                    }
                    const float minus = m == -INFINITY ? 0.f : -m;
                    const uint64_t minus2 = f2(minus, minus);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x, y;
                        f2_split(add2(f2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])),
                                      minus2),
                                 x, y);
                        w[e] = El<T>::pack(ex2(x), ex2(y));
                        sum[e & 1] = add2(sum[e & 1], El<T>::unpack(w[e]));
                    }
                    l2 = fma2(l2, f2(alpha, alpha), add2(sum[0], sum[1]));
                }
                // the step before has read its weights and written O
                ok = ok && (sc == 0 || warp_wait(bar(kPvDone), (uint32_t)((sc - 1) & 1), limit));
                fence_after();
                if (live) {
                    if (j > g.j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        const uint64_t al2 = f2(alpha, alpha);
#pragma unroll 1
                        for (int c = 0; c < R / 2; c += 32) {
                            uint32_t o[32];
                            ld32(tmem + lanes + C::COL_O + ocol + c, o);
                            ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x, y;
                                f2_split(mul2(f2(__uint_as_float(o[2 * e]),
                                                 __uint_as_float(o[2 * e + 1])),
                                              al2),
                                         x, y);
                                o[2 * e] = __float_as_uint(x);
                                o[2 * e + 1] = __float_as_uint(y);
                            }
                            st32(tmem + lanes + C::COL_O + ocol + c, o);
                        }
                        if (!C::WIDE) st_wait();
                    }
                    if (!C::WIDE) {
                        // row rl of the half's 64 tokens: 128 bytes, 16-byte piece c at
                        // c ^ (rl % 8)
                        const uint32_t p = sP + half * 8192 + rl * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            st_shared_v4(p + ((c ^ (rl & 7)) << 4), w[4 * c], w[4 * c + 1],
                                         w[4 * c + 2], w[4 * c + 3]);
                        fence_async_smem();
                    } else {
                        // over the step's scores, which both halves' warps have read
                        st32(tmem + lanes + (uint32_t)(sc & 1) * C::COL_S + half * 32, w);
                        st_wait();
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(pfull);
            }
            // the tile's output
            ok = ok && warp_wait(bar(kPvDone), (uint32_t)((sc - 1) & 1), limit);
            fence_after();
            if (live) {
                float x, y;
                f2_split(l2, x, y);
                float l = x + y;
                s_x[par][half][rl] = l;
                named_sync(1 + block, 64);
                l += s_x[par][1 - half][rl];
                par ^= 1;
                const bool mine = row < g.rows && ok;
                const int64_t slot = pair * 2 + g.slot;
                if (mine && !g.whole && half == 0)
                    a.ml[slot * a.slot_rows + row] = make_float2(m, l);
                const float inv = l > 0.f ? 1.f / l : l;     // (NaN stays NaN)
                uint16_t* orow = a.out + ((int64_t)g.q0 * a.H + g.row + row) * R + half * (R / 2);
                float* prow = a.acc + ((slot * (R / 8) + half * (R / 16)) * a.slot_rows + row) * 8;
#pragma unroll 1
                for (int c = 0; c < R / 2; c += 64) {
                    uint32_t o[64];
                    ld64(tmem + lanes + C::COL_O + ocol + c, o);
                    ld_wait(o);
                    if (!mine) continue;
                    if (g.whole) {
                        uint32_t p[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            p[e] = inv != 0.f ? El<T>::pack(__uint_as_float(o[2 * e]) * inv,
                                                            __uint_as_float(o[2 * e + 1]) * inv)
                                              : 0u;
                        if (a.out_v8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) st_global_v8(orow + c + 16 * e, p + 8 * e);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(orow + c + 8 * e) =
                                    make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            st_global_v8(prow + (int64_t)(c / 8 + e) * a.slot_rows * 8, o + 8 * e);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(oread);
            // the first part of a tile that goes on in the next pairs' runs
            if (!g.whole && g.j0 == 0 && rank == 0 && warp == 2 && lane == 0) {
                // steps of the tile from this run's end on, and the runs they fall in
                const int64_t total = s_start.total, np = min((int64_t)a.pairs, total);
                const int64_t e = run_begin(total, np, pair + 1);   // first step after this run
                const int64_t z = e + (wk.q.nt - g.j1) - 1;  // the tile's last
                int64_t last = z * np / total;               // the run that holds it
                while (last + 1 < np && run_begin(total, np, last + 1) <= z) ++last;
                while (run_begin(total, np, last) > z) --last;
                a.rec[pair] = Rec{g.q0 * a.H + g.row, ok ? g.rows : 0, pair * 2 + g.slot,
                                  (int)(last - pair) + 1};
            }
        }
        if (!ok && lane == 0) fail();
    }

    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_meet();
    if (limit->gave_up) end_given_up<C>(smem_u32(bars), smem_u32(s_used));
    if (warp == 1) {
        fence_after();
        dealloc_pair(tmem);
    }
}

// Joins the parts of a row tile: with M the largest m of a part,
//   out = sum_k 2^(m_k - M) acc_k / sum_k 2^(m_k - M) l_k
// (m: what the row's weights were formed below).
// blockIdx.x: the pair that left the first part; a block takes 8 rows and 256 elements,
// a thread 8 elements of a row, in one pass over the parts, kJoinParts of them loaded
// at a time.
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 4;

template <typename T, int R>
__global__ void __launch_bounds__(kJoinThreads) latent_decode_join(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Rec rec = a.rec[blockIdx.x];
    const int r = blockIdx.y * 8 + (threadIdx.x & 7);
    const int d = blockIdx.z * 32 + (threadIdx.x >> 3);      // eight elements
    // what a kernel that gave up left may be anything: nothing out of range
    if (r >= rec.rows || rec.rows > a.slot_rows || rec.parts < 1 || rec.slot < 0 ||
        rec.slot / 2 + rec.parts > a.pairs || rec.row0 < 0 ||
        (int64_t)rec.row0 + rec.rows > (int64_t)a.T * a.H)
        return;
    float M = -INFINITY, L = 0.f;
    float o[8] = {};
    for (int k0 = 0; k0 < rec.parts; k0 += kJoinParts) {
        float2 ml[kJoinParts];
        float4 v[kJoinParts][2];
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            if (k0 + k < rec.parts) {
                const int64_t slot = k0 + k == 0 ? rec.slot : (rec.slot / 2 + k0 + k) * 2;
                ml[k] = a.ml[slot * a.slot_rows + r];
                const float4* p = reinterpret_cast<const float4*>(
                    a.acc + ((slot * (R / 8) + d) * a.slot_rows + r) * 8);
                v[k][0] = p[0];
                v[k][1] = p[1];
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) top = fmaxf(top, ml[k].x);
        const float f0 = M == -INFINITY ? 0.f : ex2(M - top);
        M = top;
        L *= f0;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f0;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) {
            // a part without a token that the row sees: nothing, whatever its output holds
            if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
            const float f = ex2(ml[k].x - M);
            L = fmaf(f, ml[k].y, L);
            const float x[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(f, x[e], o[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : L;          // (NaN stays NaN)
    reinterpret_cast<uint4*>(a.out + ((int64_t)rec.row0 + r) * R)[d] =
        make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                   pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
}

// ------------------------------------------------------------ host side
struct Layout {
    size_t ml, acc, total;
    int rows;
};
Layout layout(int H, int R, int max_qlen, int tile) {
    Layout l;
    const int64_t rows = (int64_t)H * (max_qlen > 0 ? max_qlen : 1);
    l.rows = (int)(rows < tile ? rows : tile);
    l.ml = pkv::align_up(sizeof(Rec) * kMaxPairs, 256);
    l.acc = pkv::align_up(l.ml + 8 * (size_t)(2 * kMaxPairs) * l.rows, 256);
    l.total = l.acc + 4 * (size_t)(2 * kMaxPairs) * l.rows * R;
    return l;
}

// Rows of `row` elements in chunks of 64: boxes of `chunks` chunks of 8 rows.
bool chunk_map(CUtensorMap* m, bool bf16, const void* at, int64_t rows, int row, int chunks) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = pkv::map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(row / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)row * 2, 128};
    const cuuint32_t box[3] = {64, 8, (cuuint32_t)chunks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(at), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int R, int TILE>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const Args& a, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(latent_decode_pair<T, R, TILE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg<R, TILE>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * a.pairs));
    cfg.blockDim = dim3(Cfg<R, TILE>::THREADS);
    cfg.dynamicSmemBytes = Cfg<R, TILE>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, latent_decode_pair<T, R, TILE>, tq, tk, tv, a);
    if (e != cudaSuccess) return e;
    // (the same split of the SMs' memory as the kernel before: no change of it between)
    e = cudaFuncSetAttribute(latent_decode_join<T, R>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t jc = {};
    jc.gridDim = dim3((unsigned)a.pairs, (unsigned)((a.slot_rows + 7) / 8), R / 256);
    jc.blockDim = dim3(kJoinThreads);
    jc.stream = stream;
    jc.attrs = attr + 1;
    jc.numAttrs = 1;
    return cudaLaunchKernelEx(&jc, latent_decode_join<T, R>, a);
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
    *bytes = layout(num_heads, latent_dim, max_query_len, latent_dim == 256 ? 256 : 128).total;
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
    // the tiled copies address cache rows and query rows with 32-bit coordinates
    if (num_blocks < 1 || num_blocks > ((1LL << 31) - 65) / block_size)
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_blocks must be >= 1, and num_blocks * block_size below 2^31 - 64",
                         fn);
    if ((int64_t)num_query_tokens * num_heads > (1LL << 31) - 256)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_query_tokens * num_heads must be below 2^31 - 256",
                         fn);
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
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) ||
        !aligned(ancestors, 8))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: misaligned block_tables, context_lens, query_start or ancestors", fn);
    if (!aligned(workspace, 256))
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace must be 256-byte aligned", fn);
    // R = 256 leaves tensor memory for tiles of 256 rows: half the copies and steps where the
    // sequences' rows fill them, each step longer.  16 sequences of 1000-4000, 128 heads x 4
    // tokens: 42.3 us by 128 rows, 34.4 by 256; 32 of 20 heads x 12 42.4 and 34.8; 32 of 128
    // heads x 1 27.2 and 32.0; 33 trees of 20-260 rows, 140 on average, 31.1 (818 steps) and
    // 31.8 (515).  The width is the launch's, so it goes by the call's average.
    const bool wide = latent_dim == 256 &&
                      (int64_t)num_query_tokens * num_heads > (int64_t)192 * num_seqs;
    const int tile = wide ? 256 : 128;
    const Layout l = layout(num_heads, latent_dim, max_query_len, tile);
    if (workspace_bytes < l.total)
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace too small (%zu < %zu bytes)", fn,
                         workspace_bytes, l.total);
    const int W = latent_dim + kP;
    const int64_t rows = (int64_t)num_query_tokens * num_heads;
    if (overlap(out, rows * latent_dim * 2, q, rows * W * 2) ||
        overlap(out, rows * latent_dim * 2, cache, num_blocks * block_size * W * 2) ||
        overlap(out, rows * latent_dim * 2, workspace, (int64_t)l.total))
        return pkv::fail(PKV_ERR_INVALID, "%s: out overlaps an input or the workspace", fn);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    const int sms = pkv::sm_count(dev);
    if (sms < 2) return pkv::fail(PKV_ERR_CUDA, "%s: no multiprocessors", fn);

    const bool bf16 = dtype == PKV_BF16;
    CUtensorMap tq, tk, tv;
    const int64_t places = num_blocks * block_size;
    if (!chunk_map(&tq, bf16, q, rows, W, W / 64))
        return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of q", fn);
    if (!chunk_map(&tk, bf16, cache, places, W, latent_dim == 512 ? Cfg<512, 128>::KC : Cfg<256, 128>::KC) ||
        !chunk_map(&tv, bf16, cache, places, W, latent_dim / 128))
        return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of the cache", fn);

    Args a = {};
    a.out = static_cast<uint16_t*>(out);
    a.cache = static_cast<const uint16_t*>(cache);
    a.tables = block_tables;
    a.ctx = context_lens;
    a.q_start = query_start;
    a.ancestors = ancestors;
    a.scale_log2 = scale_log2;
    a.S = num_seqs;
    a.H = num_heads;
    a.B = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.max_qlen = max_query_len;
    a.T = num_query_tokens;
    a.num_blocks = num_blocks;
    a.slot_rows = l.rows;
    a.log_rows = wide ? 8 : 7;
    a.out_v8 = aligned(out, 32) ? 1 : 0;
    // pairs: no more than there can be steps
    int64_t pairs = sms / 2 < kMaxPairs ? sms / 2 : kMaxPairs;
    const int64_t per_seq = (((int64_t)max_blocks_per_seq * block_size + kTok - 1) / kTok) *
                            (((int64_t)max_query_len * num_heads + (1 << a.log_rows) - 1) >>
                             a.log_rows);
    if (per_seq < pairs && per_seq * num_seqs < pairs) pairs = per_seq * num_seqs;
    a.pairs = (int)pairs;
    char* ws = static_cast<char*>(workspace);
    a.rec = reinterpret_cast<Rec*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + l.ml);
    a.acc = reinterpret_cast<float*>(ws + l.acc);
    a.err = err;
    a.wait_ns = pkv::decode_wait_ns();
    if (bf16)
        e = latent_dim == 512 ? launch<__nv_bfloat16, 512, 128>(tq, tk, tv, a, stream)
            : wide            ? launch<__nv_bfloat16, 256, 256>(tq, tk, tv, a, stream)
                              : launch<__nv_bfloat16, 256, 128>(tq, tk, tv, a, stream);
    else
        e = latent_dim == 512 ? launch<__half, 512, 128>(tq, tk, tv, a, stream)
            : wide            ? launch<__half, 256, 256>(tq, tk, tv, a, stream)
                              : launch<__half, 256, 128>(tq, tk, tv, a, stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
