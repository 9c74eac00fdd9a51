// Paged decode attention for query heads that share key/value heads, with
// capped scores, a sliding window and a distance bias.
//
// What it computes, for sequence s with n tokens, query head h reading K/V
// head h / G (G = num_heads / num_kv_heads), p = n - 1:
//   z_t = scale * q[s][h] . K[t];  z_t = cap tanh(z_t / cap)  (cap > 0)
//   z_t += slope[h] (t - p)                                   (slopes given)
//   out[s][h] = sum_t softmax_t(z) V[t],   t in [lo, n), lo = max(0, n - window)
// (window 0: lo = 0), K[t] = k_cache[table[s][t / B]][h / G][t % B].
//
// Bound: the bytes of the visible K and V, each read once per K/V head; G
// query heads make 4 G D operations of 4 D bytes, which the CUDA cores cannot
// keep up with from G of about 4 on, so the products run as m16n8k16
// tensor-core products (one every 8.4 cycles per sub-core, four times what the
// memory can feed; the fifth-generation unit would add nothing but hand-offs).
//
// Design.  The work is the ordered space of steps (s, row, j): a row is a K/V
// head and up to 8 (G <= 8) or 16 of its query heads, a step ST tokens.  The
// space is cut into equal ranges, one per CTA of a persistent grid, and each
// into equal ranges for its WARPS, whatever the mix of lengths: until they are
// done, a CTA's warps share nothing.  A warp walks its range with a ring of
// kStages stages of its own.  One more warp fills the rings, a lane each: it
// walks the ring's range too, looks up the blocks of the step after the one it
// copies, and issues tiled bulk copies of whole cache rows (128-byte swizzle)
// as soon as a stage is free.  (Copies issued by the computing warps themselves
// took 900 of a step's 2100 cycles.)  Two shallow stages a warp are enough:
// deeper rings only queue up more in the memory system, where the lookups and
// queries of the next row then wait behind them.
//   S = Q K^T: the heads are the product's 16 rows, the tokens its columns;
//   online softmax in log2 units, a row's statistics in the four lanes that
//   hold it; P goes straight from S's registers to the operand of O += P V.
//   P is split into a 16-bit high part and the 16-bit residual, so weights keep
//   at least 16 bits (fp16: those above 2^-20 of the row's largest).  With up to 8
//   heads, rows 8-15 of the product are free: the residual takes them, and O is the
//   sum of row r and row r + 8 at the end, at no further product.  With 9 to 16
//   heads the residual is a second product.
// A warp ends with at most two partial rows (running max, sum, unnormalised
// output), of a row that began before its range and one that goes on after it,
// left in shared memory; the CTA joins those of the same row.  Rows that CTAs
// share leave one part in each, and a second kernel joins them.  All joins are
// in range order, so results do not vary from call to call.
//
// Measured (GB300, us a call, both kernels, and the share of the measured 6.8
// TB/s copy rate that the visible K and V come at): 8 sequences of 8192-32768
// tokens, 32/8 heads x 128, bf16, 111 us, 0.93; 64 of 1-2048, 40/8 x 128, fp16,
// capped, 50.0 us, 0.79; 33 of 17-8191, 16/1 x 64, bf16, window 1000, biased, 10.8 us; one
// of 500, 7.0 us.  About 7 us of a call do not shrink with the bytes: the ranges'
// start (lengths, tables, queries, the first copies, one behind the other) and
// the second kernel.
//
// Masked tokens (before the window, past the context) are excluded by
// selection in S, and their V rows are zeroed in shared memory, so what the
// pool holds there never matters; blocks without a visible token are neither
// copied nor looked up.
#include <cuda.h>

#include <cmath>

#include "decode_kernel.cuh"
#include "pkv_internal.h"
#include "tensor_map.h"

namespace {

using namespace pkv::dec;

constexpr int kStages = 2;                  // ring stages per warp
constexpr int kStepTokens = 16;             // tokens a step at head_dim 128, twice that at 64
constexpr int kMaxCtas = 512;
constexpr int kMinSteps = 2;                // fewest steps of a CTA
// Weights are formed as 2^(z - max + kLift), and the running max is raised only past
// a growth of kRaise (log2).  fp16 has 2^-24 as its smallest step: without the lift
// weights below 2^-25 of the largest would vanish from the product with V and stay in
// the sum of weights, which tens of thousands of them beside a large one show (32768
// of 2^-25.2: up to 0.6 of what they add to the output, 2^-11 of the values, was
// lost).  Lifted by 2^11, at most 2^15 within a raise of 4 (the roundings below keep
// that bound for scores of any size), they are held to 2^-36 of the row's largest.
template <typename T>
struct Weight {
    static constexpr float kLift = 0.f, kRaise = 8.f;
};
template <>
struct Weight<__half> {
    static constexpr float kLift = 11.f, kRaise = 4.f;
};
// Largest cap whose scores are formed as cap (1 - 2 / (2^y + 1)), which is off by
// up to 2^-20 of the CAP: up to here 2^-14 in the score, below the outputs'
// rounding.  Above it tanhf, whose error goes with the score.
constexpr float kDirectCap = 64.f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 3-D tiled bulk tensor copy global -> this CTA's shared memory, completion
// counted in bytes on `bar`.
__device__ __forceinline__ void tensor_g2s3(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// x / y of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}

// [0, n) cut into k runs of base or base + 1, the longer ones first.
struct Cut {
    int64_t base, longer;
    __device__ __forceinline__ Cut(int64_t n, int64_t k) {
        base = quotient(n, k);
        longer = n - base * k;
    }
    __device__ __forceinline__ int64_t begin(int64_t i) const {
        return i * base + (i < longer ? i : longer);
    }
    __device__ __forceinline__ int64_t run_of(int64_t x) const {
        const int64_t at = longer * (base + 1);
        return x < at ? quotient(x, base + 1) : longer + quotient(x - at, base);
    }
};

// A row split between CTAs, recorded by the one in which it begins.
struct Record {
    int s, row, last, pad;                  // s < 0: none; last: the CTA that holds its end
};

// A warp's part of a row it does not hold whole.
struct Part {
    int s, row;                             // s < 0: none
    int ended;                              // the row's last step is in the warp's range
    int last;                               // the CTA that holds the row's last step
};

// Where a warp's range begins, for the lane that fills its ring.
struct Start {
    int s, hk, gc, j, left;
};

struct Args {
    void* out;
    const void* q;
    const int32_t* tables;
    const int32_t* ctx;
    const float* slopes;
    float score;           // scale * log2(e); with a cap 2 log2(e) scale / cap, past kDirectCap scale
    float cap_log2;        // cap * log2(e); 0: no cap
    float cap_inv;         // 1 / cap past kDirectCap, else 0
    int window, S, H, HK, G, chunks, max_blocks, cap_tokens, lgB, tpc, num_blocks;
    int ctas;              // of the grid
    uint64_t wait_ns;
    Record* rec;           // [ctas]
    // parts of rows that CTAs share, two per CTA (a row that began before it,
    // one that begins in it): [2 ctas][heads a row]
    float2* ml;            // running max (log2), sum
    float* acc;            // [D]: unnormalised output
    int32_t* err;
};

template <int D, bool WIDE>
struct Geo {
    // Warps that compute, a range each: with the one that copies, 8 (225-249
    // registers) or 12 (168) of them fill the register file.
    static constexpr int WARPS = D == 64 ? 11 : 7;
    static constexpr int THREADS = WARPS * 32;          // (32 more copy)
    static constexpr int ST = kStepTokens * 128 / D;    // tokens of a step
    static constexpr int SUBS = ST / 16;
    static constexpr int HPR = WIDE ? 16 : 8;           // heads of a row
    static constexpr int HALF = ST * D * 2;             // bytes of a step's K (or V)
    static constexpr int STAGE = 2 * HALF;
    static constexpr int RING = kStages * STAGE;        // a warp's ring
    static constexpr int PART = HPR * (D + 2) * 4;      // a part: acc[HPR][D], (m, l)[HPR]
    // the parts of rows that begin in a warp take the place of its ring
    static_assert(PART <= RING && PART % 16 == 0, "part");
    static constexpr int PARTS_OFF = WARPS * RING;
    static constexpr int BAR_OFF = PARTS_OFF + WARPS * PART;
    static constexpr int CTX_OFF = BAR_OFF + 16 * WARPS * kStages;   // full, empty
    static constexpr int PREFIX_OFF = CTX_OFF + 4 * THREADS;
    static constexpr int META_OFF = (PREFIX_OFF + 4 * (THREADS + 1) + 15) / 16 * 16;
    static constexpr int START_OFF = META_OFF + 2 * WARPS * (int)sizeof(Part);
    static constexpr int SMEM = 1024 + START_OFF + WARPS * (int)sizeof(Start) + 4 * WARPS;
    static constexpr int BOXES = ST / 8;                // most boxes (block pieces) of a step
    static_assert(SMEM <= 232448, "shared memory");
};

// One sequence's tokens in steps.
struct Seq {
    int n, lo, j0, steps;
};
template <int ST>
__device__ __forceinline__ Seq seq_of(const Args& a, int c) {
    Seq q;
    q.n = c < 0 ? 0 : c > a.cap_tokens ? a.cap_tokens : c;
    q.lo = a.window > 0 && q.n > a.window ? q.n - a.window : 0;
    q.j0 = q.lo / ST;
    q.steps = q.n > 0 ? (q.n - 1) / ST + 1 - q.j0 : 0;
    return q;
}

// What a CTA's warps share: the context lengths (in shared memory where a
// thread has one sequence at most) and the steps before each thread's ones.
struct Batch {
    const int* ctx;
    const int* prefix;                      // [computing threads + 1]
    int per;                                // sequences a thread
};

// A place in the step space: step j (from 0) of the row of K/V head hk and its
// query heads' chunk gc, sequence s.
template <int ST>
struct Cursor {
    int s, hk, gc, j;
    Seq q;
    // one step on; true when that is another row
    __device__ __forceinline__ bool next(const Args& a, const Batch& b) {
        if (++j < q.steps) return false;
        j = 0;
        if (++gc < a.chunks) return true;
        gc = 0;
        if (++hk < a.HK) return true;
        hk = 0;
        do {
            ++s;
            if (s >= a.S) return true;
            q = seq_of<ST>(a, b.ctx[s]);
        } while (q.steps == 0);
        return true;
    }
};

// Step x of the space: its sequence, row and step (one warp).
template <int ST, int WARPS>
__device__ __forceinline__ Cursor<ST> locate(const Args& a, const Batch& b, int64_t x, int lane) {
    const int rows = a.HK * a.chunks;
    // the sequence holds step P of the batch counted once per sequence
    const int P = (int)quotient(x, rows);
    constexpr int kEach = WARPS;            // threads a lane
    const int g = __popc(__ballot_sync(kFull, b.prefix[lane * kEach] <= P)) - 1;
    const int t = g * kEach +
                  __popc(__ballot_sync(kFull, lane < kEach && b.prefix[g * kEach + lane % kEach] <= P)) - 1;
    int before = b.prefix[t];
    Cursor<ST> c;
    c.s = t;
    if (b.per > 1) {
        const int end = min(a.S, (t + 1) * b.per);
        for (int s0 = t * b.per; s0 < end; s0 += 32) {
            const int s = s0 + lane;
            const int n = s < end ? seq_of<ST>(a, b.ctx[s]).steps : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned hit = __ballot_sync(kFull, before + incl > P);
            if (hit) {
                const int f = __ffs(hit) - 1;
                c.s = s0 + f;
                before += __shfl_sync(kFull, incl - n, f);
                break;
            }
            before += __shfl_sync(kFull, incl, 31);
        }
    }
    c.q = seq_of<ST>(a, b.ctx[c.s]);
    const int64_t in = x - (int64_t)before * rows;
    const int row = (int)quotient(in, c.q.steps);
    c.j = (int)(in - (int64_t)row * c.q.steps);
    c.hk = a.chunks == 1 ? row : row / a.chunks;
    c.gc = row - c.hk * a.chunks;
    return c;
}

// The copies of a CTA's rings, one warp: lane i fills warp i's ring with the
// steps of its range.  Returns once every copy has been issued (or a wait for a
// free stage ran out: false), the copies themselves still in flight.
template <typename T, int D, bool WIDE>
__device__ __forceinline__ bool fill(const CUtensorMap& tk, const CUtensorMap& tv, const Args& a,
                                     const Batch& b, unsigned char* base, uint64_t* bars,
                                     const Start* starts, int& issued) {
    using C = Geo<D, WIDE>;
    constexpr int ST = C::ST, NB = C::BOXES;
    const int lane = threadIdx.x & 31, w = lane < C::WARPS ? lane : 0;
    uint64_t* full = bars + w * kStages;
    uint64_t* empty = bars + (C::WARPS + w) * kStages;
    const uint32_t ring = smem_addr(base + w * C::RING);
    const Start from = starts[w];
    const int left = lane < C::WARPS ? from.left : 0;

    Cursor<ST> c, ahead;                    // the step to copy, the one to look up
    c.s = from.s;
    c.hk = from.hk;
    c.gc = from.gc;
    c.j = from.j;
    if (left > 0) c.q = seq_of<ST>(a, b.ctx[c.s]);
    ahead = c;
    int blk[NB], next[NB];                  // physical blocks, a box each
    int looked = 0;                         // steps looked up
    auto look = [&](int (&e)[NB]) {
        if (looked >= left) return;
        const int t0 = (ahead.q.j0 + ahead.j) * ST;
        const int32_t* row = a.tables + (int64_t)ahead.s * a.max_blocks;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int tok = t0 + i * a.tpc;
            if (i * a.tpc < ST && tok < ahead.q.n && tok + a.tpc > ahead.q.lo)
                e[i] = row[tok >> a.lgB];
        }
        ++looked;
        ahead.next(a, b);
    };
    look(blk);
    look(next);
    issued = 0;
    int st = 0;
    uint32_t phase = 1;                     // of empty: the first round finds every stage free
    uint64_t since = 0;
    while (__any_sync(kFull, issued < left)) {
        const bool go = issued < left && mbar_try_wait(empty + st, phase);
        if (!__any_sync(kFull, go)) {
            const uint64_t now = global_ns();
            if (since == 0) since = now;
            if (now - since > a.wait_ns) return false;
            __nanosleep(32);
            continue;
        }
        since = 0;
        if (go) {
            const int t0 = (c.q.j0 + c.j) * ST;
            const int t1 = min(t0 + ST, c.q.n), f = max(t0, c.q.lo) & -a.tpc;
            mbar_arrive_expect_tx(full + st, (uint32_t)((t1 - f + a.tpc - 1) & -a.tpc) *
                                                 (uint32_t)(4 * D));
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int tok = t0 + i * a.tpc;
                if (i * a.tpc >= ST || tok < f || tok >= t1) continue;
                if ((unsigned)blk[i] >= (unsigned)a.num_blocks) {
                    atomicOr(a.err, PKV_DEVERR_BAD_BLOCK);
                    blk[i] = 0;                             // a valid row; flagged
                }
                const int y = ((blk[i] * a.HK + c.hk) << a.lgB) + (tok & ((1 << a.lgB) - 1));
                const uint32_t dst = ring + st * C::STAGE + i * a.tpc * (2 * D);
                tensor_g2s3(dst, &tk, 0, 0, y, full + st);
                tensor_g2s3(dst + C::HALF, &tv, 0, 0, y, full + st);
            }
            ++issued;
            c.next(a, b);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) blk[i] = next[i];
            look(next);
        }
    }
    return true;
}

// One warp's range: `left` steps from step x, at cc.  Its parts go to shared
// memory, described in meta[0] (a row that began before the range) and meta[1]
// (a row that begins in it and goes on).
template <typename T, int D, bool WIDE>
__device__ __forceinline__ void walk(const Args& a, const Batch& b, Cursor<Geo<D, WIDE>::ST> cc,
                                     const int64_t x, const int left, unsigned char* gring,
                                     unsigned char* part0, uint64_t* full, uint64_t* empty,
                                     Part* meta, const Cut& cut) {
    using C = Geo<D, WIDE>;
    constexpr int ST = C::ST, SUBS = C::SUBS, HPR = C::HPR, NH = WIDE ? 2 : 1;
    constexpr int QW = WIDE ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, kq = lane & 3;
    const uint32_t ring = smem_addr(gring);

    // a row's query fragments: head r (and r + 8), elements 16 kk + 2 kq and + 8
    auto load_q = [&](uint32_t (&qf)[D / 16][QW], const Cursor<ST>& c) {
        const int heads = min(HPR, a.G - c.gc * HPR);
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q) +
                             ((int64_t)c.s * a.H + c.hk * a.G + c.gc * HPR + r) * (D / 2) + kq;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qf[kk][0] = r < heads ? qr[kk * 8] : 0u;
            qf[kk][1] = r < heads ? qr[kk * 8 + 4] : 0u;
            if constexpr (WIDE) {
                qf[kk][2] = r + 8 < heads ? qr[kk * 8 + 8 * (D / 2)] : 0u;
                qf[kk][3] = r + 8 < heads ? qr[kk * 8 + 4 + 8 * (D / 2)] : 0u;
            }
        }
    };
    // this row's, and the next one's, loaded while this one runs
    uint32_t qa[D / 16][QW], qn[D / 16][QW];
    load_q(qn, cc);

    // Fragment addresses in a stage's K (or V): a token is D / 64 lines of 128
    // bytes, chunk c of line i at c ^ (i % 8).  Lane (mi, mr) addresses row mr of
    // the mi-th 8 x 8 matrix: K, tokens 8 (mi >> 1) + mr, chunk 2 kk + (mi & 1);
    // V, tokens 8 (mi & 1) + mr, chunk 2 c + (mi >> 1).
    const int mi = lane >> 3, mr = lane & 7;
    const int flip = D == 128 ? mr & 3 : mr >> 1, low = D == 128 ? 0 : mr & 1;
    const uint32_t krow = (uint32_t)(((mi >> 1) * 8 + mr) * (2 * D)) + (((mi & 1) ^ low) << 4);
    const uint32_t vrow = (uint32_t)(((mi & 1) * 8 + mr) * (2 * D)) + (((mi >> 1) ^ low) << 4);
    // (the second line of a token has its low chunk bit flipped)
    auto at = [&](uint32_t row, int k) -> uint32_t {
        return ((k >> 2) ? (row ^ 16u) + 128u : row) + (uint32_t)(((k & 3) ^ flip) << 5);
    };

    int st = 0;
    uint32_t phase = 0;
    bool began_before = cc.j > 0;
    for (int done = 0; done < left;) {
        const int heads = min(HPR, a.G - cc.gc * HPR);
        const int part_steps = min(left - done, cc.q.steps - cc.j);
        float m[NH], l[NH], slope[NH];
        float acc[D / 8][4];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            slope[i] = a.slopes && r + 8 * i < heads
                           ? a.slopes[cc.hk * a.G + cc.gc * HPR + r + 8 * i] * kLog2e : 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int e = 0; e < QW; ++e) qa[kk][e] = qn[kk][e];
        Cursor<ST> nc = cc;                 // the next row
        nc.j = nc.q.steps - 1;
        if (done + part_steps < left) {
            nc.next(a, b);
            load_q(qn, nc);
        }

        for (int k = 0; k < part_steps; ++k) {
            if (!__all_sync(kFull, wait_phase(full + st, phase, nullptr, a.wait_ns))) {
                if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
                return;
            }
            const int t0 = (cc.q.j0 + cc.j + k) * ST;
            const bool edge = t0 < cc.q.lo || t0 + ST > cc.q.n;
            const uint32_t sk = ring + st * C::STAGE, sv = sk + C::HALF;
            if (edge) {
                // V rows of hidden tokens
                for (int i = lane; i < ST * (D / 8); i += 32) {
                    const int tok = t0 + i / (D / 8);
                    if (tok < cc.q.lo || tok >= cc.q.n)
                        *reinterpret_cast<uint4*>(gring + st * C::STAGE + C::HALF + i * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }

            // z[u][v][2 i + e]: head r + 8 i, token t0 + 16 u + 8 v + 2 kq + e
            float z[SUBS][2][4];
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[u][0][e] = z[u][1][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int u = 0; u < SUBS; ++u) {
                    uint32_t kb[4];
                    ldsm_x4(kb, sk + u * (16 * 2 * D) + at(krow, kk));
                    const uint32_t af[4] = {qa[kk][0], WIDE ? qa[kk][QW - 2] : 0u, qa[kk][1],
                                            WIDE ? qa[kk][QW - 1] : 0u};
                    mma16816<T>(z[u][0], af, kb[0], kb[1]);
                    mma16816<T>(z[u][1], af, kb[2], kb[3]);
                }
            auto each = [&](auto f) {
#pragma unroll
                for (int u = 0; u < SUBS; ++u)
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int i = 0; i < NH; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                f(z[u][v][2 * i + e], t0 + u * 16 + v * 8 + 2 * kq + e, i);
            };
            each([&](float& y, int, int) { y *= a.score; });
            if (a.cap_inv > 0.f)
                each([&](float& y, int, int) { y = a.cap_log2 * tanhf(y * a.cap_inv); });
            else if (a.cap_log2 > 0.f)      // cap tanh(y) = cap (1 - 2 / (2^(2 log2(e) y) + 1))
                each([&](float& y, int, int) {
                    y = a.cap_log2 * (1.f - __fdividef(2.f, ex2(y) + 1.f));
                });
            if (a.slopes)
                each([&](float& y, int t, int i) { y += slope[i] * (float)(t - (cc.q.n - 1)); });
            if (edge)
                each([&](float& y, int t, int) {
                    if (t < cc.q.lo || t >= cc.q.n) y = -INFINITY;
                });
            float mx[NH], alpha[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) mx[i] = -INFINITY;
            each([&](float& y, int, int i) { mx[i] = fmaxf(mx[i], y); });
            bool raised = false;
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 2));
                const bool up = mx[i] > __fadd_rd(m[i], Weight<T>::kRaise) || m[i] == -INFINITY;
                alpha[i] = up ? ex2(m[i] - mx[i]) : 1.f;
                if (up) m[i] = mx[i];
                raised |= up;
            }
            if (__any_sync(kFull, raised)) {
#pragma unroll
                for (int i = 0; i < NH; ++i) l[i] *= alpha[i];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    acc[i][0] *= alpha[0];
                    acc[i][1] *= alpha[0];
                    acc[i][2] *= alpha[NH - 1];
                    acc[i][3] *= alpha[NH - 1];
                }
            }
            float top[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) top[i] = __fadd_ru(m[i], -Weight<T>::kLift);
            each([&](float& y, int, int i) { y = ex2(y - top[i]); });
            if (edge)                       // (m is -infinity where every visible score is)
                each([&](float& y, int t, int) {
                    if (t < cc.q.lo || t >= cc.q.n) y = 0.f;
                });
            each([&](float& y, int, int i) { l[i] += y; });
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                uint32_t hi[2][NH], lo[2][NH];
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int i = 0; i < NH; ++i) {
                        const float p0 = z[u][v][2 * i], p1 = z[u][v][2 * i + 1];
                        hi[v][i] = pack2<T>(p0, p1);
                        const float2 h = unpack2<T>(hi[v][i]);
                        lo[v][i] = pack2<T>(p0 - h.x, p1 - h.y);
                    }
                const uint32_t pa[4] = {hi[0][0], WIDE ? hi[0][NH - 1] : lo[0][0], hi[1][0],
                                        WIDE ? hi[1][NH - 1] : lo[1][0]};
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t vb[4];
                    ldsm_x4_t(vb, sv + u * (16 * 2 * D) + at(vrow, c));
                    mma16816<T>(acc[2 * c], pa, vb[0], vb[1]);
                    mma16816<T>(acc[2 * c + 1], pa, vb[2], vb[3]);
                    if constexpr (WIDE) {
                        const uint32_t pl[4] = {lo[0][0], lo[0][NH - 1], lo[1][0], lo[1][NH - 1]};
                        mma16816<T>(acc[2 * c], pl, vb[0], vb[1]);
                        mma16816<T>(acc[2 * c + 1], pl, vb[2], vb[3]);
                    }
                }
            }
            // the stage is free: its values are in registers (and a zeroed row
            // is written before the next copy lands over it)
            if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }

        // the row's part in this range ends here
        done += part_steps;
        const bool row_end = cc.j + part_steps == cc.q.steps;
        const bool whole = row_end && !began_before;
        // (a row that goes on is the warp's last: every copy has landed and been
        // read, so its part may take the ring's place)
        unsigned char* part = began_before ? part0 : gring;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            float sum = l[i];
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            const int hr = r + 8 * i;
            if (hr >= heads) continue;
            const float inv = 1.f / sum;
            uint32_t* o = reinterpret_cast<uint32_t*>(a.out) +
                          ((int64_t)cc.s * a.H + cc.hk * a.G + cc.gc * HPR + hr) * (D / 2) + kq;
            float2* pa = reinterpret_cast<float2*>(part) + hr * (D / 2) + kq;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const float o0 = WIDE ? acc[c][2 * i] : acc[c][0] + acc[c][2];
                const float o1 = WIDE ? acc[c][2 * i + 1] : acc[c][1] + acc[c][3];
                if (whole) o[c * 4] = pack2<T>(o0 * inv, o1 * inv);
                else pa[c * 4] = make_float2(o0, o1);
            }
            if (!whole && kq == 0)
                reinterpret_cast<float2*>(part + HPR * D * 4)[hr] = make_float2(m[i], sum);
        }
        if (!whole && lane == 0) {
            Part p;
            p.s = cc.s;
            p.row = cc.hk * a.chunks + cc.gc;
            p.ended = row_end;
            p.last = row_end ? 0 : (int)cut.run_of(x + done - 1 + (cc.q.steps - cc.j - part_steps));
            meta[began_before ? 0 : 1] = p;
        }
        began_before = false;
        cc = nc;
    }
}

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(Geo<D, WIDE>::THREADS + 32, 1)
    grouped_decode_main(const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const Args a) {
    using C = Geo<D, WIDE>;
    constexpr int ST = C::ST, HPR = C::HPR;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::BAR_OFF);
    int* ctx = reinterpret_cast<int*>(base + C::CTX_OFF);
    int* prefix = reinterpret_cast<int*>(base + C::PREFIX_OFF);
    Part* parts = reinterpret_cast<Part*>(base + C::META_OFF);   // of warp i: 2 i, 2 i + 1
    Start* starts = reinterpret_cast<Start*>(base + C::START_OFF);
    int* sums = reinterpret_cast<int*>(starts + C::WARPS);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool copies = warp == C::WARPS;
    const int c = (int)blockIdx.x;
    if (copies && lane == 0) {
        prefetch_map(&tk);
        prefetch_map(&tv);
    }
    if (!copies && lane < 2 * kStages) mbar_init(bars + lane / kStages * (C::WARPS * kStages) +
                                                 warp * kStages + lane % kStages, 1);
    if (!copies) fence_mbar_init();
    if (!copies && lane < 2) parts[2 * warp + lane].s = -1;
    grid_dependency_wait();

    // steps before each thread's sequences
    Batch b;
    b.per = (a.S + C::THREADS - 1) / C::THREADS;
    b.prefix = prefix;
    b.ctx = b.per > 1 ? a.ctx : ctx;
    int incl = 0;
    if (!copies) {
        int local = 0;
        for (int s = tid * b.per; s < a.S && s < (tid + 1) * b.per; ++s) {
            const int n = a.ctx[s];
            if (b.per == 1) ctx[tid] = n;
            local += seq_of<ST>(a, n).steps;
            if ((n < 0 || n > a.cap_tokens) && c == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
        }
        incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
    }
    __syncthreads();
    if (!copies) {
#pragma unroll
        for (int i = 0; i < C::WARPS; ++i)
            if (i < warp) incl += sums[i];
        prefix[tid + 1] = incl;
        if (tid == 0) prefix[0] = 0;
    }
    __syncthreads();
    grid_launch_dependents();

    // this CTA's run of the steps, this warp's run of it
    const int64_t X = (int64_t)(a.HK * a.chunks) * prefix[C::THREADS];
    const int64_t most = X / kMinSteps > 1 ? X / kMinSteps : 1;
    const int64_t used = X == 0 ? 0 : most < a.ctas ? most : a.ctas;
    bool recorded = false;
    if (c < used) {
        const Cut cut(X, used);
        const int64_t cx = cut.begin(c);
        const int cn = (int)(cut.begin(c + 1) - cx);
        const int each = cn / C::WARPS, longer = cn - each * C::WARPS;
        const int64_t x = cx + warp * each + min(warp, longer);
        const int left = copies ? 0 : each + (warp < longer);
        Cursor<ST> at;
        if (left > 0) at = locate<ST, C::WARPS>(a, b, x, lane);
        if (!copies && lane == 0) starts[warp] = {at.s, at.hk, at.gc, at.j, left};
        __syncthreads();
        if (copies) {
            int issued = 0;
            if (!fill<T, D, WIDE>(tk, tv, a, b, base, bars, starts, issued)) {
                if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
            }
            // let every copy land before the CTA can end, whatever the others did
            for (int g = issued - kStages < 0 ? 0 : issued - kStages; g < issued; ++g)
                wait_phase(bars + lane * kStages + g % kStages, (uint32_t)((g / kStages) & 1),
                           nullptr, kWaitLimitNs);
        } else if (left > 0) {
            walk<T, D, WIDE>(a, b, at, x, left, base + warp * C::RING,
                             base + C::PARTS_OFF + warp * C::PART, bars + warp * kStages,
                             bars + (C::WARPS + warp) * kStages, parts + 2 * warp, cut);
        }
        __syncthreads();

        // Join the parts of each row, a head of a row a warp: a row begins with
        // an odd part, or with the CTA's first where it began in an earlier CTA.
        constexpr int V = D / 32;
        const Part mine = parts[lane < 2 * C::WARPS ? lane : 0];
        const unsigned held = __ballot_sync(kFull, lane < 2 * C::WARPS && mine.s >= 0);
        const unsigned ends = __ballot_sync(kFull, lane < 2 * C::WARPS && mine.s >= 0 && mine.ended);
        unsigned begins = held & 0xaaaaaaaau;
        if (held) begins |= held & (0u - held);
        for (int unit = 0; begins; begins &= begins - 1) {
            const int first = __ffs(begins) - 1;
            const unsigned from = held & (~0u << first), end = ends & (~0u << first);
            const unsigned set = end ? from & (2u * (end & (0u - end)) - 1u) : from;
            const bool starts_here = (first & 1) != 0;
            const int s = __shfl_sync(kFull, mine.s, first);
            const int row = __shfl_sync(kFull, mine.row, first);
            if (starts_here && !end) {
                recorded = true;
                if (lane == first && warp == 0) a.rec[c] = {s, row, mine.last, 0};
            }
            const int hk = a.chunks == 1 ? row : row / a.chunks, gc = row - hk * a.chunks;
            const int heads = min(HPR, a.G - gc * HPR);
            for (int h = warp - unit % C::WARPS; h < heads; h += C::WARPS) {
                if (h < 0 || copies) continue;
                auto part = [&](int k) -> const unsigned char* {
                    return base + (k & 1 ? (k >> 1) * C::RING : C::PARTS_OFF + (k >> 1) * C::PART);
                };
                // two parts at a time: most rows here have no more
                float M = -INFINITY, L = 0.f, o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = 0.f;
                for (unsigned to_do = set; to_do;) {
                    const int k0 = __ffs(to_do) - 1;
                    to_do &= to_do - 1;
                    const bool two = to_do != 0;
                    const int k1 = two ? __ffs(to_do) - 1 : k0;
                    to_do &= to_do - 1;
                    const unsigned char *p0 = part(k0), *p1 = part(k1);
                    const float2 m0 = reinterpret_cast<const float2*>(p0 + HPR * D * 4)[h];
                    float2 m1 = reinterpret_cast<const float2*>(p1 + HPR * D * 4)[h];
                    const float* v0 = reinterpret_cast<const float*>(p0) + h * D + lane * V;
                    const float* v1 = reinterpret_cast<const float*>(p1) + h * D + lane * V;
                    if (!two) m1 = make_float2(-INFINITY, 0.f);
                    const float top = fmaxf(M, fmaxf(m0.x, m1.x));
                    const float f = k0 == first ? 0.f : ex2(M - top);
                    const float f0 = ex2(m0.x - top), f1 = two ? ex2(m1.x - top) : 0.f;
                    M = top;
                    L = L * f + m0.y * f0 + m1.y * f1;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = o[e] * f + v0[e] * f0 + v1[e] * f1;
                }
                if (starts_here && end) {
                    const float inv = __fdividef(1.f, L);
                    uint32_t* out = reinterpret_cast<uint32_t*>(a.out) +
                                    ((int64_t)s * a.H + hk * a.G + gc * HPR + h) * (D / 2) +
                                    lane * (V / 2);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e)
                        out[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
                } else {
                    const int64_t to = (2 * (int64_t)c + (starts_here ? 1 : 0)) * HPR + h;
                    float* p = a.acc + to * D + lane * V;
#pragma unroll
                    for (int e = 0; e < V; ++e) p[e] = o[e];
                    if (lane == 0) a.ml[to] = make_float2(M, L);
                }
            }
            unit += heads;
        }
    }
    if (!recorded && tid == 0) a.rec[c].s = -1;

    // rows that attend nothing
    const int64_t row_words = (int64_t)a.H * D / 8;
    for (int s = c; s < a.S; s += gridDim.x) {
        if (b.ctx[s] > 0) continue;
        uint4* o = static_cast<uint4*>(a.out) + s * row_words;
        for (int64_t i = tid; i < row_words; i += C::THREADS + 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Joins the parts of the rows that CTAs share: with M the largest running max,
//   out = sum_k 2^(m_k - M) acc_k / sum_k 2^(m_k - M) l_k.
// A CTA per recording CTA and head; its warps take every fourth part each,
// kBatch of them in flight.
constexpr int kJoinWarps = 4;

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32) grouped_decode_join(const Args a) {
    constexpr int HPR = WIDE ? 16 : 8, V = D / 32, kBatch = 8;
    __shared__ float o_[kJoinWarps][D];
    __shared__ float2 ml_[kJoinWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x, h = blockIdx.y;
    const Record rec = a.rec[c];
    if (rec.s < 0) return;
    const int hk = rec.row / a.chunks, gc = rec.row - hk * a.chunks;
    if (h >= min(HPR, a.G - gc * HPR)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = rec.last - c + 1;
    float M = -INFINITY, L = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int k0 = warp; k0 < n; k0 += kBatch * kJoinWarps) {
        float2 ml[kBatch];
        float v[kBatch][V];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + i * kJoinWarps;
            const int64_t at = (2 * (int64_t)(c + k) + (k == 0)) * HPR + h;
            ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = 0.f;
            if (k < n) {
                ml[i] = a.ml[at];
                const float* p = a.acc + at * D + lane * V;
                if constexpr (V == 4) {
                    const float4 w = *reinterpret_cast<const float4*>(p);
                    v[i][0] = w.x;
                    v[i][1] = w.y;
                    v[i][2] = w.z;
                    v[i][3] = w.w;
                } else {
                    const float2 w = *reinterpret_cast<const float2*>(p);
                    v[i][0] = w.x;
                    v[i][1] = w.y;
                }
            }
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
        // (nothing so far weighs nothing, whatever the maxima)
        const float f0 = M == -INFINITY ? 0.f : ex2(M - top);
        M = top;
        L *= f0;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= f0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float f = k0 + i * kJoinWarps < n ? ex2(ml[i].x - M) : 0.f;
            L += f * ml[i].y;
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] += f * v[i][e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) o_[warp][lane * V + e] = o[e];
    if (lane == 0) ml_[warp] = make_float2(M, L);
    __syncthreads();
    const int warps = n < kJoinWarps ? n : kJoinWarps;
    for (int d = threadIdx.x; d < D / 2; d += kJoinWarps * 32) {
        float top = -INFINITY, s0 = 0.f, s1 = 0.f, sum = 0.f;
        for (int i = 0; i < warps; ++i) top = fmaxf(top, ml_[i].x);
        for (int i = 0; i < warps; ++i) {
            const float f = ex2(ml_[i].x - top);
            s0 += f * o_[i][2 * d];
            s1 += f * o_[i][2 * d + 1];
            sum += f * ml_[i].y;
        }
        const int64_t head = (int64_t)hk * a.G + gc * HPR + h;
        reinterpret_cast<uint32_t*>(a.out)[((int64_t)rec.s * a.H + head) * (D / 2) + d] =
            pack2<T>(s0 / sum, s1 / sum);
    }
}

template <typename T, int D, bool WIDE>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Args& a, int grid,
                   cudaStream_t stream) {
    const size_t smem = Geo<D, WIDE>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(grouped_decode_main<T, D, WIDE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Geo<D, WIDE>::THREADS + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, grouped_decode_main<T, D, WIDE>, tk, tv, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)grid, WIDE ? 16 : 8);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, grouped_decode_join<T, D, WIDE>, a);
}

template <typename T>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Args& a, int D, bool wide,
                   int grid, cudaStream_t stream) {
    if (D == 64)
        return wide ? launch<T, 64, true>(tk, tv, a, grid, stream)
                    : launch<T, 64, false>(tk, tv, a, grid, stream);
    return wide ? launch<T, 128, true>(tk, tv, a, grid, stream)
                : launch<T, 128, false>(tk, tv, a, grid, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks shared by the workspace query and the launch, and the sizes that
// follow: query heads a row, rows per K/V head, the most CTAs.
struct Shape {
    int G, heads, chunks, ctas;
};
pkv_status shape_of(const char* fn, int S, int H, int HK, int D, int B, int max_blocks, Shape* out) {
    if (S < 0 || S > PKV_MAX_SEQS)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, %d]", fn, PKV_MAX_SEQS);
    if (HK < 1 || H < 1 || H > 65535 || H % HK != 0)
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_heads must be a multiple of num_kv_heads, at most 65535", fn);
    if (D != 64 && D != 128) return pkv::fail(PKV_ERR_INVALID, "%s: head_dim must be 64 or 128", fn);
    if (B != 8 && B != 16 && B != 32 && B != 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    if (max_blocks < 1) return pkv::fail(PKV_ERR_INVALID, "%s: max_blocks_per_seq must be >= 1", fn);
    if ((int64_t)max_blocks * B > (1LL << 30))
        return pkv::fail(PKV_ERR_INVALID, "%s: context capacity above 2^30 tokens", fn);
    const int st = kStepTokens * 128 / D;
    const int64_t steps = (int64_t)S * (((int64_t)max_blocks * B + st - 1) / st);
    if (steps >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: batch too large (step count overflows)", fn);
    out->G = H / HK;
    out->heads = out->G <= 8 ? 8 : 16;
    out->chunks = (out->G + out->heads - 1) / out->heads;
    if (steps * HK * out->chunks >= (1LL << 36))
        return pkv::fail(PKV_ERR_INVALID, "%s: batch too large (step count overflows)", fn);
    const int64_t most = steps * HK * out->chunks / kMinSteps;
    out->ctas = (int)(most < 1 ? 1 : most < kMaxCtas ? most : kMaxCtas);
    return PKV_OK;
}

struct Layout {
    size_t ml, acc, total;
};
Layout layout_of(const Shape& s, int D) {
    Layout l;
    const size_t rows = 2 * (size_t)s.ctas * s.heads;
    l.ml = pkv::align_up(sizeof(Record) * (size_t)s.ctas, 256);
    l.acc = pkv::align_up(l.ml + 8 * rows, 256);
    l.total = pkv::align_up(l.acc + 4 * rows * D, 256);
    return l;
}

}  // namespace

extern "C" {

pkv_status pkv_decode_grouped_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                             int head_dim, int block_size, int max_blocks_per_seq,
                                             size_t* bytes) {
    const char* fn = "pkv_decode_grouped_workspace_size";
    if (!bytes) return pkv::fail(PKV_ERR_INVALID, "%s: bytes is NULL", fn);
    Shape s;
    const pkv_status st = shape_of(fn, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                   max_blocks_per_seq, &s);
    if (st != PKV_OK) return st;
    *bytes = layout_of(s, head_dim).total;
    return PKV_OK;
}

pkv_status pkv_paged_attention_decode_grouped(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const float* slopes, float scale,
    float softcap, int window, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int64_t num_blocks, pkv_dtype dtype, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
    const char* fn = "pkv_paged_attention_decode_grouped";
    Shape sh;
    pkv_status st = shape_of(fn, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                             max_blocks_per_seq, &sh);
    if (st != PKV_OK) return st;
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    if (!std::isfinite(scale)) return pkv::fail(PKV_ERR_INVALID, "%s: scale is not finite", fn);
    if (!(softcap >= 0.f) || !std::isfinite(softcap))
        return pkv::fail(PKV_ERR_INVALID, "%s: softcap must be finite and not negative", fn);
    const double log2e = 1.4426950408889634;
    const float score = (float)(softcap > 0.f ? 2.0 * log2e * scale / softcap : log2e * scale);
    const float cap_log2 = (float)(log2e * softcap);
    if (!std::isfinite(score) || !std::isfinite(cap_log2))
        return pkv::fail(PKV_ERR_INVALID, "%s: scale and softcap are too far apart", fn);
    const bool large_cap = softcap > kDirectCap;
    if (window < 0) return pkv::fail(PKV_ERR_INVALID, "%s: window must not be negative", fn);
    // the tiled copies address cache rows (block, head, token) with 32-bit coordinates
    if (num_blocks < 1 || num_blocks > ((1LL << 31) - 1) / ((int64_t)num_kv_heads * block_size))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_blocks must be >= 1, and num_blocks * num_kv_heads * block_size "
                         "below 2^31",
                         fn);
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !workspace)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q and the caches must be 16-byte aligned", fn);
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(slopes, 4))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: block_tables, context_lens and slopes must be 4-byte aligned", fn);
    if (!aligned(workspace, 256))
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace must be 256-byte aligned", fn);
    const Layout lay = layout_of(sh, head_dim);
    if (workspace_bytes < lay.total)
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace too small (%zu < %zu bytes)", fn,
                         workspace_bytes, lay.total);

    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    const int sms = pkv::sm_count(dev);
    int32_t* err = pkv::device_error_word();
    if (sms < 1 || !err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);
    // one wave, no more CTAs than the batch could have work for
    int grid = sms;
    if (grid > sh.ctas) grid = sh.ctas;

    CUtensorMap tk, tv;
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    const int step = kStepTokens * 128 / head_dim;
    const int box = block_size < step ? block_size : step;
    if (!pkv::row_map(&tk, dtype == PKV_BF16, k_cache, rows, head_dim, box) ||
        !pkv::row_map(&tv, dtype == PKV_BF16, v_cache, rows, head_dim, box))
        return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of the caches", fn);

    char* ws = static_cast<char*>(workspace);
    Args a;
    a.out = out;
    a.q = q;
    a.tables = block_tables;
    a.ctx = context_lens;
    a.slopes = slopes;
    a.score = large_cap ? scale : score;
    a.cap_log2 = cap_log2;
    a.cap_inv = large_cap ? (float)(1.0 / softcap) : 0.f;
    a.window = window;
    a.S = num_seqs;
    a.H = num_heads;
    a.HK = num_kv_heads;
    a.G = sh.G;
    a.chunks = sh.chunks;
    a.max_blocks = max_blocks_per_seq;
    a.cap_tokens = max_blocks_per_seq * block_size;
    a.lgB = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    a.tpc = box;
    a.ctas = grid;
    a.num_blocks = (int)num_blocks;
    a.wait_ns = pkv::decode_wait_ns();
    a.rec = reinterpret_cast<Record*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + lay.ml);
    a.acc = reinterpret_cast<float*>(ws + lay.acc);
    a.err = err;
    const bool wide = sh.heads == 16;
    e = dtype == PKV_F16 ? launch<__half>(tk, tv, a, head_dim, wide, grid, stream)
                         : launch<__nv_bfloat16>(tk, tv, a, head_dim, wide, grid, stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
