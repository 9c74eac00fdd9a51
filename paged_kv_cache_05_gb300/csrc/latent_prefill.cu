// Attention of prompts in the expanded form of latent attention: a head's keys are N
// elements of its own and 64 that all heads share, its values N elements.  Query row i
// of a sequence (of qlen rows and klen keys) sees the keys t <= klen - qlen + i:
//   z_t = scale (q[0 .. N) . k_t + q[N ..) . r_t),
//   out = sum_t 2^(z_t - m) v_t / sum_t 2^(z_t - m)
// in log2 units, with the running max and sum of the softmax (one pass over the keys).
//
// Bound: the tensor cores: 2 (2 N + 64) operations a (row, key) pair of a head, against
// one exponential.  An item is 512 query rows of one head, its steps 64 keys each.  The
// products are pairs' (clusters of two CTAs, cta_group::2, M = 256): each CTA holds 128
// rows of each of two slots (rows 0-255 and 256-511 of the item) and half of a step's
// keys and values (32 keys; N / 2 elements of every value), so that a step's 40 KB come
// to the SMs once for 512 rows.  (One CTA with 256 rows alone would need 31 bytes a
// cycle of them, of the 36 that the copies reach, and read 128 bytes a cycle of its
// shared memory, all there are: 96 here.)
//
// Thirteen warps a CTA: keys, values and queries a warp each (the last walks the run and
// hands its items to the others through shared memory), one that issues the products for
// the scores and one for the outputs (the first CTA's), and four of softmax a slot, a
// thread a row.  A slot's scores S go round two places in tensor memory (N = 64: three, as
// its outputs leave room: chunks 82.4 -> 81.2 us): a step's are formed while the one before
// is weighed.  (With steps of 128 keys and one place a slot, S waits for P V of the step
// before, which waits for its softmax: 3150 cycles a step of 512 rows, where the products
// take 2560.)  Weights P are written over the scores.  The max is raised only past a growth
// of kRescale, so that most steps leave O alone.
//
// Measured (graph of calls, the joining kernel counted): 4 prompts of 1965-2036, 32 heads of
// 128, bf16: 148 us (1108 TFLOP/s; calls on changing inputs 159 us); 4 chunks of 373-541 after
// about 4100, 16 heads of 64, fp16: 80 us; one prompt of 61, 16 heads of 128: 7.1 us.  A step
// of 512 rows takes 1480 cycles with N = 64: a softmax warp's chain of loads, mask, max,
// weights, stores and hand-offs, not its arithmetic (without the exponentials N = 128 takes
// as long).
//
// The steps of all items are dealt to the pairs in equal runs; parts of an item are left
// in the workspace and joined by a second kernel.  Where no item has more than
// kWholeSteps steps, items stay whole and there is no second kernel.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
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
constexpr int kRows = 512;            // rows of an item: two slots of a pair's 256
constexpr int kKeys = 64;             // keys of a step
constexpr int kThreads = 416;
constexpr int kMaxPairs = 96;
constexpr int kWholeSteps = 8;
constexpr int kBoxRows = 16;          // keys, or values, of a box
constexpr int kQBoxRows = 32;

template <int N>
struct Cfg {
    static constexpr int CH = (N + kP) / 64;          // chunks of 64 elements of a key
    static constexpr int KS = N == 128 ? 6 : 8;       // stages
    static constexpr int VS = KS;
    // tensor memory: S (and P over it) at 64 (PL slot + place), then each slot's O
    static constexpr int PL = N == 128 ? 2 : 3;
    static constexpr uint32_t COL_O = 128 * PL;
    static_assert(COL_O + 2 * N <= 512, "tensor memory");
    static constexpr int Q_CHUNK = 128 * 128;         // a slot's rows of a chunk
    static constexpr int Q_SLOT = CH * Q_CHUNK;
    static constexpr int K_CHUNK = kKeys / 2 * 128;   // a CTA's keys of a chunk
    static constexpr int K_STAGE = CH * K_CHUNK;
    static constexpr int V_STAGE = kKeys * 128;       // 64 elements (N = 64: 32 and zeros)
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = 2 * Q_SLOT;
    static constexpr int V_OFF = K_OFF + KS * K_STAGE;
    static constexpr int SMEM = V_OFF + VS * V_STAGE + 1024;   // 1 KiB of alignment slack
    static_assert(SMEM + 2048 <= 232448, "shared memory");
};

enum : int {
    kQFull = 0,      // + slot: its rows are there (first CTA's barrier)
    kQEmpty = 2,     // + slot: an item's last S formed
    kKFull = 4,      // + stage (up to 8)
    kKEmpty = 12,    // + stage
    kVFull = 20,     // + stage
    kVEmpty = 28,    // + stage
    kSFull = 36,     // + PL slot + place: S formed
    kPFull = 42,     // + PL slot + place: weights written, O rescaled (first CTA's)
    kPvDone = 48,    // + PL slot + place: P V done
    kORead = 54,     // + slot: its output read from tensor memory (first CTA's)
    kItFull = 56,    // + entry (4)
    kItEmpty = 60,   // + entry
    kBars = 64
};

struct Args {
    uint16_t* out;
    const uint16_t* v;
    int64_t v_stride, v_head;
    const int32_t *q_start, *k_start;
    float scale_log2;                 // above 0
    int negative;                     // the scale is below: scores of -q
    int S, H, max_q, max_k, Tq, Tk;
    int pairs, slot_rows;             // rows of a part in the workspace
    int out_v8;                       // out is 32-byte aligned: 32-byte stores
    int whole;                        // items stay whole
    struct Rec* rec;                  // [pairs]
    float2* ml;                       // [2 pairs][slot_rows]
    float* acc;                       // [2 pairs][N / 8][slot_rows][8]
    int32_t* err;
    uint64_t wait_ns;                 // of a wait (pkv_set_decode_wait_limit)
};

// What is left to join: rows of the output of a head whose parts lie in `parts` slots:
// `slot`, then the first of each following pair.
struct Rec {
    int row0, rows, head, slot, parts, pad[3];
};

struct Seq {
    int q0, k0, qlen, klen;           // qlen 0: nothing to do
    // what a sequence's lengths are, as they lie in memory ...
    __device__ __forceinline__ void fetch(const Args& a, int s) {
        q0 = a.q_start[s];
        qlen = a.q_start[s + 1];
        k0 = a.k_start[s];
        klen = a.k_start[s + 1];
    }
    // ... and looked at (the loads are waited for here)
    __device__ __forceinline__ bool look(const Args& a) {
        qlen -= q0;
        klen -= k0;
        if (qlen < 0 || qlen > a.max_q || q0 < 0 || (int64_t)q0 + qlen > a.Tq || klen < qlen ||
            klen > a.max_k || k0 < 0 || (int64_t)k0 + klen > a.Tk) {
            qlen = 0;
            return false;
        }
        return true;
    }
    __device__ __forceinline__ bool load(const Args& a, int s) {
        fetch(a, s);
        return look(a);
    }
    __device__ __forceinline__ int items() const { return (qlen + kRows - 1) / kRows; }
    // steps of item t: to the key of its last row
    __device__ __forceinline__ int steps(int t) const {
        return (klen - qlen + min(qlen, (t + 1) * kRows) + kKeys - 1) / kKeys;
    }
    __device__ __forceinline__ int64_t head_steps() const {
        int64_t n = 0;
        for (int t = 0; t < items(); ++t) n += steps(t);
        return n;
    }
};

// Where a pair's run begins.
struct Start {
    int s;
    Seq q;
    int64_t off, n;                   // steps before it in the sequence, steps of the run
    int64_t total;                    // steps of all
};

// Steps [j0, j1) of an item.  Slot 0's rows see fewer of the last steps' keys: up to step
// `both` the two slots work, then one alone.  An item of 256 rows or fewer has one slot,
// the other than the one before it had.
struct Item {
    int q0, k0, klen, h;              // first row of all, first key of all
    int off;                          // the last key that its row 0 sees
    int rows;                         // 0: no more items
    int j0, j1, steps;                // (steps: of the whole item)
    int both, alone;                  // j0 <= both <= j1; the slot that is then alone
    int row1, live0, live1;           // slot 1's first row, each slot's rows
    int slot;                         // of a part: 0 the run's first, 1 another
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == steps; }
    // a slot's steps are [j0, end)
    __device__ __forceinline__ int end(int x) const { return x == alone ? j1 : both; }
};
constexpr int kRing = 4;              // items on their way from the warp that walks the run

struct Walker {
    Seq q, next;
    int s, h, t, j;
    int64_t left;
    int turn;                         // the slot of the next item that has one
    bool first;
    __device__ __forceinline__ void init(const Args& a, const Start& st) {
        s = st.s;
        q = st.q;
        left = st.n;
        first = true;
        turn = 0;
        h = t = j = 0;
        if (left <= 0) return;
        if (s + 1 < a.S) next.fetch(a, s + 1);
        const int64_t per = q.head_steps();
        h = per < (1 << 30) && st.off < (1 << 30) ? (int)st.off / (int)per : (int)(st.off / per);
        int64_t rest = st.off - h * per;
        while (rest >= q.steps(t)) rest -= q.steps(t++);
        j = (int)rest;
        if (a.whole && j > 0) {                       // the run's items are those that begin in it
            left -= q.steps(t) - j;
            j = 0;
            ++t;
        }
    }
    __device__ __forceinline__ bool get(const Args& a, Item& it) {
        if (left <= 0) return false;
        while (t >= q.items()) {
            t = 0;
            if (q.qlen > 0 && ++h < a.H) break;
            h = 0;
            if (++s >= a.S) return false;
            q = next;
            q.look(a);
            if (s + 1 < a.S) next.fetch(a, s + 1);
        }
        it.q0 = q.q0 + t * kRows;
        it.k0 = q.k0;
        it.klen = q.klen;
        it.h = h;
        it.off = q.klen - q.qlen + t * kRows;
        it.rows = min(kRows, q.qlen - t * kRows);
        it.steps = q.steps(t);
        it.j0 = j;
        it.j1 = a.whole ? it.steps : (int)min((int64_t)it.steps, j + left);
        if (it.rows > kRows / 2) {
            // slot 0's rows end earlier
            it.both = max(min((it.off + kRows / 2 + kKeys - 1) / kKeys, it.j1), j);
            it.alone = 1;
            turn = 0;
        } else {
            it.both = j;
            it.alone = turn;
            turn ^= 1;
        }
        if (it.rows > kRows / 2) {
            it.row1 = it.live0 = kRows / 2;
            it.live1 = it.rows - kRows / 2;
        } else {
            it.row1 = 0;
            it.live0 = it.alone == 0 ? it.rows : 0;
            it.live1 = it.alone == 1 ? it.rows : 0;
        }
        it.slot = first ? 0 : 1;
        first = false;
        left -= it.j1 - it.j0;
        j = 0;
        if (it.j1 == it.steps) ++t;
        return true;
    }
};

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
        copies(kKFull, C::KS);
        copies(kVFull, C::VS);
        for (int x = 0; x < 2; ++x) {
            products(kSFull + C::PL * x, C::PL);
            products(kPvDone + C::PL * x, C::PL);
            products(kQEmpty + x, 1);
            copies(kQFull + x, 1);
        }
    }
    fence_before();
    __syncthreads();
    cluster_sync();
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_pair(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_r,
                        const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using C = Cfg<N>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ uint32_t s_tmem;
    __shared__ Limit s_limit;
    __shared__ int s_used[kBars];                   // phases of a ring, at its first barrier's place
    __shared__ Start s_start;
    __shared__ Item s_items[kRing];
    __shared__ int64_t s_scan[2][kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = (int)(blockIdx.x >> 1);
    volatile Limit* const limit = &s_limit;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sQ = base + C::Q_OFF, sK = base + C::K_OFF, sV = base + C::V_OFF;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the pair's run of the steps: [b, e) of all (the lengths are loaded once where
    // there is a thread a sequence, and on their way while the barriers are made)
    Seq mine;
    mine.qlen = 0;
    bool good = tid >= a.S || mine.load(a, tid);
    if (warp == 1) {
        for (int i = lane; i < kBars; i += 32) {
            const bool two = i < kQEmpty || (i >= kKFull && i < kKEmpty) ||
                             (i >= kVFull && i < kVEmpty);
            const bool warps = (i >= kPFull && i < kPvDone) || i == kORead || i == kORead + 1;
            // an item's readers: keys, values, eight of softmax, the two of products
            const int n = two ? 2 : warps ? 8 : i >= kItEmpty ? (rank ? 10 : 12) : 1;
            mbar_init(bar(i), n);
        }
        mbar_init_fence();
        for (int i = lane; i < kBars; i += 32) s_used[i] = kNotCounted;
        if (lane == 0) s_limit = Limit{a.wait_ns, 0};
        __syncwarp();
        alloc_pair(smem_u32(&s_tmem));
    } else if (warp == 0 && lane == 0) {
        prefetch_map(&tm_q);
        prefetch_map(&tm_k);
        prefetch_map(&tm_r);
        prefetch_map(&tm_v);
    }
    {
        constexpr int kWarps = kThreads / 32;
        // this thread's steps, and those of the threads before it in the warp
        int64_t n = mine.head_steps() * a.H, incl = n, rest = 0;
        for (int s = tid + kThreads; s < a.S; s += kThreads) {
            Seq q;
            good &= q.load(a, s);
            rest += q.head_steps() * a.H;
        }
        if (!good && blockIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (a.S > kThreads) {
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) incl += s_scan[0][w];
            before += s_scan[0][w];
            total += s_scan[0][w] + s_scan[1][w];
        }
        const int64_t np = min((int64_t)a.pairs, total);
        const int64_t b = pair < np ? run_begin(total, np, pair) : 0;
        const int64_t e = pair < np ? run_begin(total, np, pair + 1) : 0;
        auto found = [&](int s) {                // the sequence that holds step b
            if (e > b && incl > b && incl - n <= b)
                s_start = Start{s, mine, b - (incl - n), e - b, total};
        };
        found(tid);
        for (int s0 = kThreads; s0 < a.S && before <= b && e > b; s0 += kThreads) {
            mine.qlen = 0;
            if (s0 + tid < a.S) mine.load(a, s0 + tid);
            n = incl = mine.head_steps() * a.H;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) s_scan[0][warp] = incl;
            __syncthreads();
            incl += before;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) incl += s_scan[0][w];
                before += s_scan[0][w];
            }
            found(s0 + tid);
        }
        // (nothing to join, until a part is left)
        if (tid == 0 && rank == 0 && !a.whole) a.rec[pair].rows = 0;
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

    // the next item of the run, from the warp that walks it
    int items = 0;
    auto next_item = [&](Item& it) {
        const int e = items % kRing;
        ok = ok && warp_wait(bar(kItFull + e), (uint32_t)((items / kRing) & 1), limit);
        it = s_items[e];
        __syncwarp();
        // (one that gave up hands nothing back: others may not have read the entry)
        if (ok && lane == 0) mbar_arrive(bar(kItEmpty + e));
        ++items;
        return ok && it.rows > 0;
    };
    auto next_alone = [&](Item& it) {            // (by one thread)
        const int e = items % kRing;
        ok = ok && mbar_wait<false>(bar(kItFull + e), (uint32_t)((items / kRing) & 1), limit);
        it = s_items[e];
        if (ok) mbar_arrive(bar(kItEmpty + e));
        ++items;
        return ok && it.rows > 0;
    };
    if (warp == 0) {
        // ================================================= keys
        Item it;
        int kc = 0;
        constexpr int BOXES = kKeys / 2 / kBoxRows;
        const int c = lane / BOXES, r = (lane - c * BOXES) * kBoxRows;   // a lane's box
        while (next_item(it)) {
            for (int j = it.j0; j < it.j1; ++j, ++kc) {
                const int st = kc % C::KS, n = kc / C::KS;
                if (n > 0 && !warp_wait(bar(kKEmpty + st), (uint32_t)((n - 1) & 1), limit)) {
                    ok = false;
                    break;
                }
                const uint32_t full = at_rank(bar(kKFull + st), 0);
                if (lane == 0) mbar_expect_tx_relaxed(full, C::K_STAGE);
                __syncwarp();
                const uint32_t to = sK + st * C::K_STAGE + c * C::K_CHUNK + r * 128;
                const int key = it.k0 + j * kKeys + kKeys / 2 * (int)rank + r;
                if (c < C::CH - 1) tma_3d_pair(to, &tm_k, c * 64, it.h, key, full);
                else if (c == C::CH - 1) tma_3d_pair(to, &tm_r, 0, 0, key, full);
            }
        }
        // (the products' last releases arrive before the CTA ends: see cluster_meet)
        ok = ok && ring_ended(bar(kKEmpty), C::KS, kc, limit);
        if (!ok) {
            if (lane == 0) s_used[kKFull] = kc;
            fail();
        }
    } else if (warp == 2) {
        // ================================================= values
        Item it;
        int vc = 0;
        constexpr int BOXES = kKeys / kBoxRows;
        while (next_item(it)) {
            for (int j = it.j0; j < it.j1; ++j, ++vc) {
                const int st = vc % C::VS, n = vc / C::VS;
                if (n > 0 && !warp_wait(bar(kVEmpty + st), (uint32_t)((n - 1) & 1), limit)) {
                    ok = false;
                    break;
                }
                const uint32_t full = at_rank(bar(kVFull + st), 0);
                const uint32_t stage = sV + st * C::V_STAGE;
                const int left = it.klen - j * kKeys;        // keys of the step and after
                // the box that holds the sequence's last key and others' rows behind it,
                // which may be anything: copied by the warp, zeros behind the last
                const int tail = left < kKeys && left % kBoxRows ? left / kBoxRows : -1;
                if (tail >= 0) {
                    const uint16_t* from = a.v + (int64_t)(it.k0 + j * kKeys + tail * kBoxRows) * a.v_stride +
                                           it.h * a.v_head + (int)rank * (N / 2);
                    uint4 w[kBoxRows / 4];
#pragma unroll
                    for (int e = 0; e < kBoxRows / 4; ++e) {
                        const int r = 4 * e + (lane >> 3), p = lane & 7;
                        w[e] = make_uint4(0u, 0u, 0u, 0u);
                        if (r < left % kBoxRows && p < N / 16)
                            w[e] = *reinterpret_cast<const uint4*>(from + r * a.v_stride + p * 8);
                    }
#pragma unroll
                    for (int e = 0; e < kBoxRows / 4; ++e) {
                        const int r = 4 * e + (lane >> 3), p = lane & 7;
                        st_shared_v4(stage + (tail * kBoxRows + r) * 128 + ((p ^ (r & 7)) << 4), w[e].x,
                                     w[e].y, w[e].z, w[e].w);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    if (tail >= 0) mbar_expect_tx_cluster(full, C::V_STAGE - kBoxRows * 128);
                    else mbar_expect_tx_relaxed(full, C::V_STAGE);
                }
                __syncwarp();
                // boxes behind the last key: past the tensor's end, zeros
                if (lane < BOXES && lane != tail)
                    tma_3d_pair(stage + lane * kBoxRows * 128, &tm_v, (int)rank * (N / 2), it.h,
                                lane * kBoxRows < left ? it.k0 + j * kKeys + lane * kBoxRows : a.Tk,
                                full);
            }
        }
        ok = ok && ring_ended(bar(kVEmpty), C::VS, vc, limit);
        if (!ok) {
            if (lane == 0) s_used[kVFull] = vc;
            fail();
        }
    } else if (warp == 3) {
        // ================================================= items and queries
        Walker wk;
        wk.init(a, start);
        Item it;
        int count[2] = {0, 0};
        constexpr int BOXES = 128 / kQBoxRows;
        const int c = lane / BOXES, r = (lane - c * BOXES) * kQBoxRows;
        for (int n = 0; ok; ++n) {
            const bool more = wk.get(a, it);
            if (!more) it.rows = 0;
            const int e = n % kRing;
            if (n >= kRing && !warp_wait(bar(kItEmpty + e), (uint32_t)((n / kRing - 1) & 1), limit)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                s_items[e] = it;
                mbar_arrive(bar(kItFull + e));
            }
            if (!more) break;
            for (int x = 0; x < 2; ++x) {
                if (it.end(x) <= it.j0) continue;
                const int n = count[x];
                if (n > 0 && !warp_wait(bar(kQEmpty + x), (uint32_t)((n - 1) & 1), limit)) {
                    ok = false;
                    break;
                }
                const uint32_t full = at_rank(bar(kQFull + x), 0);
                if (lane == 0) mbar_expect_tx_relaxed(full, C::Q_SLOT);
                __syncwarp();
                if (c < C::CH)
                    tma_3d_pair(sQ + x * C::Q_SLOT + c * C::Q_CHUNK + r * 128, &tm_q, c * 64, it.h,
                                it.q0 + (x ? it.row1 : 0) + 128 * (int)rank + r, full);
                ++count[x];
            }
        }
        for (int x = 0; x < 2; ++x) ok = ok && ring_ended(bar(kQEmpty + x), 1, count[x], limit);
        if (!ok) {
            if (lane == 0) {
                s_used[kQFull] = count[0];
                s_used[kQFull + 1] = count[1];
            }
            fail();
        }
    } else if (warp == 1) {
        // ================================================= scores
        if (rank == 0 && elect_one()) {
            const uint32_t ID_S = idesc(El<T>::kType, false, kKeys, 256) | (a.negative ? kNegateA : 0);
            const uint64_t dQ = sdesc(sQ, 16, 1024), dK = sdesc(sK, 16, 1024);
            Item it;
            int g = 0, n[2] = {0, 0};        // steps of the run, of each slot
            int ends[2] = {0, 0};            // items of each slot whose scores are all formed
            uint32_t qs = 0;                 // a slot's phase of its queries, by bits
            while (next_alone(it)) {
                for (int j = it.j0; ok && j < it.j1; ++j, ++g) {
                    const int st = g % C::KS;
                    ok = mbar_wait<false>(bar(kKFull + st), (uint32_t)((g / C::KS) & 1), limit);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!ok || j >= it.end(x)) continue;
                        if (j == it.j0) {
                            ok = mbar_wait<false>(bar(kQFull + x), qs >> x & 1, limit);
                            qs ^= 1u << x;
                        }
                        // the place is free once P V of the step that had it is done
                        const int p = n[x] % C::PL;
                        if (ok && n[x] >= C::PL)
                            ok = mbar_wait<false>(bar(kPvDone + C::PL * x + p),
                                                  (uint32_t)(n[x] / C::PL - 1) & 1, limit);
                        if (!ok) continue;
                        fence_after();
                        const uint64_t da = dQ + (uint64_t)((x * C::Q_SLOT) >> 4);
                        const uint64_t db = dK + (uint64_t)((st * C::K_STAGE) >> 4);
#pragma unroll
                        for (int e = 0; e < C::CH * 4; ++e)
                            umma_pair(tmem + (C::PL * x + p) * 64,
                                      da + (((e >> 2) * C::Q_CHUNK + (e & 3) * 32) >> 4),
                                      db + (((e >> 2) * C::K_CHUNK + (e & 3) * 32) >> 4), ID_S, e > 0);
                        commit_pair(bar(kSFull + C::PL * x + p));
                        if (j == it.end(x) - 1) {
                            commit_pair(bar(kQEmpty + x));
                            ++ends[x];
                        }
                        ++n[x];
                    }
                    // (a stage whose copy may be on its way is never handed back)
                    if (!ok) break;
                    commit_pair(bar(kKEmpty + st));
                }
            }
            s_used[kKEmpty] = g;
            for (int x = 0; x < 2; ++x) {
                s_used[kSFull + C::PL * x] = n[x];
                s_used[kQEmpty + x] = ends[x];
            }
            if (!ok) fail();
        }
        __syncwarp();
    } else if (warp == 12) {
        // ================================================= outputs
        if (rank == 0 && elect_one()) {
            constexpr uint32_t ID_PV = idesc(El<T>::kType, true, N, 256);
            const uint64_t dV = sdesc(sV, 1024, 1024);
            Item it;
            int g = 0, n[2] = {0, 0};        // steps of the run, of each slot
            uint32_t left = 0, os = 0;       // by bits: slots that left an output, its phase
            while (next_alone(it)) {
                for (int j = it.j0; ok && j < it.j1; ++j, ++g) {
                    const int st = g % C::VS;
                    ok = mbar_wait<false>(bar(kVFull + st), (uint32_t)((g / C::VS) & 1), limit);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!ok || j >= it.end(x)) continue;
                        const int p = n[x] % C::PL;
                        ok = mbar_wait<false>(bar(kPFull + C::PL * x + p),
                                              (uint32_t)(n[x] / C::PL) & 1, limit);
                        if (ok && j == it.j0 && (left >> x & 1)) {
                            ok = mbar_wait<false>(bar(kORead + x), os >> x & 1, limit);
                            os ^= 1u << x;
                        }
                        if (!ok) continue;
                        fence_after();
                        const uint64_t db = dV + (uint64_t)((st * C::V_STAGE) >> 4);
#pragma unroll
                        for (int e = 0; e < kKeys / 16; ++e)
                            umma_ts_pair(tmem + C::COL_O + x * N, tmem + (C::PL * x + p) * 64 + e * 8,
                                         db + ((e * 2048) >> 4), ID_PV, j > it.j0 || e > 0);
                        commit_pair(bar(kPvDone + C::PL * x + p));
                        left |= 1u << x;
                        ++n[x];
                    }
                    if (!ok) break;
                    commit_pair(bar(kVEmpty + st));
                }
            }
            // the last outputs' readers, of both CTAs, have arrived before this one ends
            for (int x = 0; x < 2; ++x)
                if (ok && (left >> x & 1))
                    ok = mbar_wait<false>(bar(kORead + x), os >> x & 1, limit);
            s_used[kVEmpty] = g;
            for (int x = 0; x < 2; ++x) s_used[kPvDone + C::PL * x] = n[x];
            if (!ok) fail();
        }
        __syncwarp();
    } else {
        // ================================================= softmax
        const int x = warp >= 8, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tO = tmem + lanes + C::COL_O + x * N;
        const uint32_t pfull = at_rank(bar(kPFull + C::PL * x), 0), oread = at_rank(bar(kORead + x), 0);
        Item it;
        int n = 0;                           // steps of this slot
        const uint64_t scale2 = f2(a.scale_log2, a.scale_log2);
        while (next_item(it)) {
            const int at = (int)rank * 128 + quad * 32;      // the warp's first row of the slot's
            const int mine_rows = x ? it.live1 : it.live0;
            const bool live = at < mine_rows;
            const int rw = (x ? it.row1 : 0) + at, row = rw + lane;      // and of the item's
            const int64_t slot = pair * 2 + it.slot;
            const int end = it.end(x);
            const bool whole = it.whole();
            // the row's weights are 2^(z - m), its scores z at most m + kLift + kRescale:
            // m is the largest so far, or a little less, lowered by the lift
            float m = -INFINITY;
            uint64_t l2 = 0;                                 // two partial sums
            for (int j = it.j0; j < end; ++j, ++n) {
                const int place = n % C::PL;
                const uint32_t tS = tmem + lanes + (C::PL * x + place) * 64;
                ok = ok && warp_wait(bar(kSFull + C::PL * x + place), (uint32_t)(n / C::PL) & 1,
                                     limit);
                fence_after();
                if (live) {
                    uint32_t z[64];
                    ld64(tS, z);
                    ld_wait(z);
                    if (it.off + rw + 1 - j * kKeys < kKeys) {
                        const int seen = it.off + row + 1 - j * kKeys;
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= seen) z[e] = __float_as_uint(-INFINITY);
                    }
                    float top = __uint_as_float(z[0]), t1 = __uint_as_float(z[1]);
#pragma unroll
                    for (int e = 2; e < 62; e += 4) {
                        top = max3(top, __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
                        t1 = max3(t1, __uint_as_float(z[e + 2]), __uint_as_float(z[e + 3]));
                    }
                    top = fmaxf(max3(top, __uint_as_float(z[62]), __uint_as_float(z[63])), t1);
                    top = fabsf(top) == INFINITY ? -INFINITY : __fmul_rn(top, a.scale_log2);
                    // the scores, scaled and rounded as the largest was: in one operation with
                    // its subtraction, what its rounding left, up to half a step of a large
                    // score, would be in every weight
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float p, q;
                        f2_split(mul2(f2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])),
                                      scale2),
                                 p, q);
                        z[2 * e] = __float_as_uint(p);
                        z[2 * e + 1] = __float_as_uint(q);
                    }
                    float alpha = 1.f;
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
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p, q;
                            f2_split(add2_rz(f2(__uint_as_float(z[32 * c + 2 * e]),
                                                __uint_as_float(z[32 * c + 2 * e + 1])),
                                             minus2),
                                     p, q);
                            p = ex2(p);
                            q = ex2(q);
                            sum[e & 1] = add2(sum[e & 1], f2(p, q));
                            w[e] = El<T>::pack(p, q);
                        }
                        st16(tS + c * 16, w);
                    }
                    l2 = fma2(l2, f2(alpha, alpha), add2(sum[0], sum[1]));
                    if (j > it.j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        // P V of the step before has to be in O
                        ok = ok && warp_wait(bar(kPvDone + C::PL * x + (n - 1) % C::PL),
                                             (uint32_t)((n - 1) / C::PL) & 1, limit);
                        fence_after();
                        const uint64_t al2 = f2(alpha, alpha);
#pragma unroll 1
                        for (int c = 0; c < N; c += 32) {
                            uint32_t o[32];
                            ld32(tO + c, o);
                            ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float p, q;
                                f2_split(mul2(f2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])),
                                              al2),
                                         p, q);
                                o[2 * e] = __float_as_uint(p);
                                o[2 * e + 1] = __float_as_uint(q);
                            }
                            st32(tO + c, o);
                        }
                    }
                    st_wait();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(pfull + place * 8);
            }
            // the slot's output
            float p, q;
            f2_split(l2, p, q);
            const float l = p + q;
            const bool mine = at + lane < mine_rows && ok;
            if (mine && !whole) a.ml[slot * a.slot_rows + row] = make_float2(m, l);
            if (end > it.j0) {
                ok = ok && warp_wait(bar(kPvDone + C::PL * x + (n - 1) % C::PL),
                                     (uint32_t)((n - 1) / C::PL) & 1, limit);
                fence_after();
                if (live) {
                    const float inv = 1.f / l;
                    uint16_t* orow = a.out + ((int64_t)(it.q0 + row) * a.H + it.h) * N;
                    float* prow = a.acc + (slot * (N / 8) * a.slot_rows + row) * 8;
                    uint32_t next[32];
                    ld32(tO, next);
#pragma unroll 1
                    for (int c = 0; c < N; c += 32) {
                        uint32_t o[32];
                        ld_wait(next);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = next[e];
                        if (c + 32 < N) ld32(tO + c + 32, next);
                        if (!mine) continue;
                        if (whole) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = El<T>::pack(__uint_as_float(o[2 * e]) * inv,
                                                   __uint_as_float(o[2 * e + 1]) * inv);
                            if (a.out_v8) {
                                st_global_v8(orow + c, w);
                                st_global_v8(orow + c + 16, w + 8);
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    *reinterpret_cast<uint4*>(orow + c + 8 * e) =
                                        make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                st_global_v8(prow + (int64_t)(c / 8 + e) * a.slot_rows * 8, o + 8 * e);
                        }
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(oread);
            }
            // the first part of an item that goes on in the next pairs' runs
            if (!whole && it.j0 == 0 && rank == 0 && warp == 4 && lane == 0) {
                const int64_t total = s_start.total, np = min((int64_t)a.pairs, total);
                const int64_t e = run_begin(total, np, pair + 1);   // first step after this run
                const int64_t z = e + (it.steps - it.j1) - 1;    // the item's last
                int64_t last = z * np / total;               // the run that holds it
                while (last + 1 < np && run_begin(total, np, last + 1) <= z) ++last;
                while (run_begin(total, np, last) > z) --last;
                a.rec[pair] = Rec{it.q0, ok ? it.rows : 0, it.h, pair * 2 + it.slot,
                                  (int)(last - pair) + 1, {0, 0, 0}};
            }
        }
        ok = ok && ring_ended(bar(kPvDone + C::PL * x), C::PL, n, limit);
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

// Joins the parts of an item: with M the largest m of a part,
//   out = sum_k 2^(m_k - M) acc_k / sum_k 2^(m_k - M) l_k
// (m: what the row's weights were formed below).
// blockIdx.x: the pair that left the first part; a block takes 8 rows and 256 / 8
// eights of elements (N = 64: 32 rows), a thread 8 elements of a row, in one pass over
// the parts, kJoinParts of them loaded at a time.
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 4;

template <typename T, int N>
__global__ void __launch_bounds__(kJoinThreads) latent_prefill_join(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsAtOnce = kJoinThreads / (N / 8);
    const Rec rec = a.rec[blockIdx.x];
    const int r = blockIdx.y * kRowsAtOnce + (int)threadIdx.x % kRowsAtOnce;
    const int d = threadIdx.x / kRowsAtOnce;                 // eight elements
    // what a kernel that gave up left may be anything: nothing out of range
    if (r >= rec.rows || rec.rows > a.slot_rows || rec.parts < 1 || rec.slot < 0 ||
        rec.slot / 2 + rec.parts > a.pairs || rec.row0 < 0 || rec.head < 0 || rec.head >= a.H ||
        (int64_t)rec.row0 + rec.rows > a.Tq)
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
                    a.acc + ((slot * (N / 8) + d) * a.slot_rows + r) * 8);
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
            // a part without a key that the row sees: nothing, whatever its output holds
            if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
            const float f = ex2(ml[k].x - M);
            L = fmaf(f, ml[k].y, L);
            const float x[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(f, x[e], o[e]);
        }
    }
    const float inv = 1.f / L;
    reinterpret_cast<uint4*>(a.out + (((int64_t)rec.row0 + r) * a.H + rec.head) * N)[d] =
        make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                   pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
}

// ------------------------------------------------------------ host side
struct Layout {
    size_t ml, acc, total;
    int rows;
};
Layout layout(int N, int max_q, int max_k) {
    Layout l = {};
    if (max_k <= kWholeSteps * kKeys) return l;       // items stay whole
    l.rows = max_q < kRows ? (max_q > 0 ? max_q : 1) : kRows;
    l.ml = pkv::align_up(sizeof(Rec) * kMaxPairs, 256);
    l.acc = pkv::align_up(l.ml + 8 * (size_t)(2 * kMaxPairs) * l.rows, 256);
    l.total = l.acc + 4 * (size_t)(2 * kMaxPairs) * l.rows * N;
    return l;
}

// Tokens of heads of `row` elements, as boxes of 64 elements of box_rows tokens of a head.
bool head_map(CUtensorMap* m, bool bf16, const void* at, int row, int heads, int64_t tokens,
              int64_t token_stride, int64_t head_stride, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = pkv::map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)row, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(at), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int N>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tr,
                   const CUtensorMap& tv, const Args& a, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(latent_prefill_pair<T, N>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<N>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * a.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<N>::SMEM;
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
    e = cudaLaunchKernelEx(&cfg, latent_prefill_pair<T, N>, tq, tk, tr, tv, a);
    if (e != cudaSuccess || a.whole) return e;
    // (the same split of the SMs' memory as the kernel before: no change of it between)
    e = cudaFuncSetAttribute(latent_prefill_join<T, N>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t jc = {};
    constexpr int kRowsAtOnce = kJoinThreads / (N / 8);
    jc.gridDim = dim3((unsigned)a.pairs, (unsigned)((a.slot_rows + kRowsAtOnce - 1) / kRowsAtOnce));
    jc.blockDim = dim3(kJoinThreads);
    jc.stream = stream;
    jc.attrs = attr + 1;
    jc.numAttrs = 1;
    return cudaLaunchKernelEx(&jc, latent_prefill_join<T, N>, a);
}

}  // namespace

extern "C" {

pkv_status pkv_latent_prefill_workspace_size(int head_dim, int max_query_len, int max_key_len,
                                             size_t* bytes) {
    const char* fn = "pkv_latent_prefill_workspace_size";
    if (!bytes) return pkv::fail(PKV_ERR_INVALID, "%s: bytes is NULL", fn);
    if ((head_dim != 64 && head_dim != 128) || max_query_len < 0 || max_key_len < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    *bytes = layout(head_dim, max_query_len, max_key_len).total;
    return PKV_OK;
}

pkv_status pkv_latent_attention_prefill(
    void* out, const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
    int64_t k_stride, int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
    const void* v, int64_t v_stride, int64_t v_head_stride, const int32_t* query_start,
    const int32_t* key_start, float scale, int num_seqs, int num_heads, int head_dim, int rope_dim,
    int max_query_len, int max_key_len, int num_query_tokens, int num_key_tokens, pkv_dtype dtype,
    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
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
    // the tiled copies address tokens with 32-bit coordinates
    if (num_query_tokens > (1 << 30) || num_key_tokens > (1 << 30))
        return pkv::fail(PKV_ERR_INVALID, "%s: at most 2^30 tokens", fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    const float scale_log2 = (float)(1.4426950408889634 * scale);
    if (!std::isfinite(scale_log2))
        return pkv::fail(PKV_ERR_INVALID, "%s: scale is not finite", fn);
    const struct {
        const void* at;
        int64_t token, head, row, heads, tokens;
        const char* name;
    } in[4] = {{q, q_stride, q_head_stride, head_dim + kP, num_heads, num_query_tokens, "q"},
               {k, k_stride, k_head_stride, head_dim, num_heads, num_key_tokens, "k"},
               {k_rope, k_rope_stride, kP, kP, 1, num_key_tokens, "k_rope"},
               {v, v_stride, v_head_stride, head_dim, num_heads, num_key_tokens, "v"}};
    for (const auto& x : in)
        if (x.token < x.row || x.head < x.row || x.token % 8 != 0 || x.head % 8 != 0 ||
            x.token > (1LL << 32) || x.head > (1LL << 32))
            return pkv::fail(PKV_ERR_INVALID,
                             "%s: strides of %s must cover a row, be multiples of 8 elements and "
                             "at most 2^32",
                             fn, x.name);
    if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PKV_OK;
    // (without keys, no sequence may have a row: the kernel looks at that)
    if (!out || !q || !query_start || !key_start || (num_key_tokens > 0 && (!k || !k_rope || !v)))
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(k_rope, 16) ||
        !aligned(v, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q, k, k_rope and v must be 16-byte aligned",
                         fn);
    if (!aligned(query_start, 4) || !aligned(key_start, 4))
        return pkv::fail(PKV_ERR_INVALID, "%s: misaligned query_start or key_start", fn);
    const int64_t out_bytes = (int64_t)num_query_tokens * num_heads * head_dim * 2;
    for (const auto& x : in)
        if (x.tokens > 0 &&
            overlap(out, out_bytes, x.at,
                    ((x.tokens - 1) * x.token + (x.heads - 1) * x.head + x.row) * 2))
            return pkv::fail(PKV_ERR_INVALID, "%s: out overlaps %s", fn, x.name);
    const Layout l = layout(head_dim, max_query_len, max_key_len);
    if (l.total > 0) {
        if (!workspace || !aligned(workspace, 256))
            return pkv::fail(PKV_ERR_INVALID, "%s: workspace must be 256-byte aligned, not NULL", fn);
        if (workspace_bytes < l.total)
            return pkv::fail(PKV_ERR_INVALID, "%s: workspace too small (%zu < %zu bytes)", fn,
                             workspace_bytes, l.total);
        if (overlap(out, out_bytes, workspace, (int64_t)l.total))
            return pkv::fail(PKV_ERR_INVALID, "%s: out overlaps the workspace", fn);
    }
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    const int sms = pkv::sm_count(dev);
    if (sms < 2) return pkv::fail(PKV_ERR_CUDA, "%s: no multiprocessors", fn);

    const bool bf16 = dtype == PKV_BF16;
    CUtensorMap tq, tk, tr, tv;
    const int64_t keys = num_key_tokens > 0 ? num_key_tokens : 1;
    if (num_key_tokens == 0) k = v = k_rope = q;      // (maps of something, never used)
    if (!head_map(&tq, bf16, q, head_dim + kP, num_heads, num_query_tokens, q_stride, q_head_stride,
                  kQBoxRows) ||
        !head_map(&tk, bf16, k, head_dim, num_heads, keys, k_stride, k_head_stride, kBoxRows) ||
        !head_map(&tv, bf16, v, head_dim, num_heads, keys, v_stride, v_head_stride, kBoxRows) ||
        !head_map(&tr, bf16, k_rope, kP, 1, keys, k_rope_stride, kP, kBoxRows))
        return pkv::fail(PKV_ERR_CUDA, "%s: tensor maps", fn);

    Args a = {};
    a.out = static_cast<uint16_t*>(out);
    a.v = static_cast<const uint16_t*>(v);
    a.v_stride = v_stride;
    a.v_head = v_head_stride;
    a.q_start = query_start;
    a.k_start = key_start;
    // (a hidden score is infinite and stays so under any scale but 0)
    a.scale_log2 = scale_log2 == 0.f ? FLT_MIN : std::fabs(scale_log2);
    a.negative = scale_log2 < 0.f;
    a.S = num_seqs;
    a.H = num_heads;
    a.max_q = max_query_len;
    a.max_k = max_key_len;
    a.Tq = num_query_tokens;
    a.Tk = num_key_tokens;
    a.out_v8 = aligned(out, 32) ? 1 : 0;
    a.whole = l.total == 0;
    a.slot_rows = l.rows;
    // pairs: no more than there can be steps (items, where they stay whole)
    int64_t pairs = sms / 2 < kMaxPairs ? sms / 2 : kMaxPairs;
    const int64_t items = (int64_t)num_seqs * num_heads * ((max_query_len + kRows - 1) / kRows);
    const int64_t each = a.whole ? 1 : ((int64_t)max_key_len + kKeys - 1) / kKeys;
    if (items < pairs && items * each < pairs) pairs = items * each;
    a.pairs = (int)pairs;
    char* ws = static_cast<char*>(workspace);
    a.rec = reinterpret_cast<Rec*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + l.ml);
    a.acc = reinterpret_cast<float*>(ws + l.acc);
    a.err = err;
    a.wait_ns = pkv::decode_wait_ns();
    if (bf16)
        e = head_dim == 128 ? launch<__nv_bfloat16, 128>(tq, tk, tr, tv, a, stream)
                            : launch<__nv_bfloat16, 64>(tq, tk, tr, tv, a, stream);
    else
        e = head_dim == 128 ? launch<__half, 128>(tq, tk, tr, tv, a, stream)
                            : launch<__half, 64>(tq, tk, tr, tv, a, stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
