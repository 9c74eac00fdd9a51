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
// kStages stages of its own, into which it issues tiled bulk copies of whole
// cache rows (128-byte swizzle) kStages steps ahead, one mbarrier a stage.
//   S = Q K^T: the heads are the product's 16 rows, the tokens its columns;
//   online softmax in log2 units, a row's statistics in the four lanes that
//   hold it; P goes straight from S's registers to the operand of O += P V.
//   P is split into a 16-bit high part and the 16-bit residual, so weights keep
//   at least 16 bits.  With up to 8 heads, rows 8-15 of the product are free:
//   the residual takes them, and O is the sum of row r and row r + 8 at the
//   end, at no further product.  With 9 to 16 heads the residual is a second
//   product.
// A warp ends with at most two partial rows (running max, sum, unnormalised
// output), of a row that began before its range and one that goes on after it,
// left in shared memory; the CTA joins those of the same row.  Rows that CTAs
// share leave one part in each, and a second kernel joins them.  All joins are
// in range order, so results do not vary from call to call.
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

#ifndef PKV_GW
#define PKV_GW 8
#endif
#ifndef PKV_GS
#define PKV_GS 2
#endif
#ifndef PKV_GT
#define PKV_GT 16
#endif
#ifndef PKV_GM
#define PKV_GM 8
#endif
constexpr int kWarps = PKV_GW;                   // ranges per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kStages = PKV_GS;                  // ring stages per warp
constexpr int kStepTokens = PKV_GT;              // tokens a step at head_dim 128, twice that at 64
constexpr int kMaxCtas = 512;
constexpr int kMinSteps = PKV_GM;                // fewest steps of a CTA
constexpr float kRaiseLog2 = 8.f;           // raise the running max only past this growth
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

struct Args {
    void* out;
    const void* q;
    const int32_t* tables;
    const int32_t* ctx;
    const float* slopes;
    float score;           // without a cap: scale * log2(e), else 2 log2(e) scale / cap
    float cap_log2;        // cap * log2(e); 0: no cap
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
    static constexpr int ST = kStepTokens * 128 / D;    // tokens of a step
    static constexpr int SUBS = ST / 16;
    static constexpr int HPR = WIDE ? 16 : 8;           // heads of a row
    static constexpr int HALF = ST * D * 2;             // bytes of a step's K (or V)
    static constexpr int STAGE = 2 * HALF;
    static constexpr int RING = kStages * STAGE;        // a warp's ring
    static constexpr int PART = HPR * (D + 2) * 4;      // a part: acc[HPR][D], (m, l)[HPR]
    // the parts of rows that begin in a warp take the place of its ring
    static_assert(PART <= RING && PART % 16 == 0, "part");
    static constexpr int PARTS_OFF = kWarps * RING;
    static constexpr int BAR_OFF = PARTS_OFF + kWarps * PART;
    static constexpr int CTX_OFF = BAR_OFF + 8 * kWarps * kStages;
    static constexpr int PREFIX_OFF = CTX_OFF + 4 * kThreads;
    static constexpr int META_OFF = (PREFIX_OFF + 4 * (kThreads + 1) + 15) / 16 * 16;
    static constexpr int SMEM = 1024 + META_OFF + 2 * kWarps * (int)sizeof(Part) + 4 * kWarps;
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
    const int* prefix;                      // [kThreads + 1]
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
template <int ST>
__device__ __forceinline__ Cursor<ST> locate(const Args& a, const Batch& b, int64_t x, int lane) {
    const int rows = a.HK * a.chunks;
    // the sequence holds step P of the batch counted once per sequence
    const int P = (int)quotient(x, rows);
    constexpr int kEach = kThreads / 32;
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
    c.hk = row / a.chunks;
    c.gc = row - c.hk * a.chunks;
    return c;
}

// One warp's range: the steps [x, x + left).  Its parts go to shared memory,
// described in meta[0] (a row that began before the range) and meta[1] (a row
// that begins in it and goes on).
template <typename T, int D, bool WIDE>
__device__ __forceinline__ void walk(const CUtensorMap& tk, const CUtensorMap& tv, const Args& a,
                                     const Batch& b, const int64_t x, const int left,
                                     unsigned char* gring, unsigned char* part0, uint64_t* full,
                                     Part* meta, const Cut& cut) {
    using C = Geo<D, WIDE>;
    constexpr int ST = C::ST, SUBS = C::SUBS, HPR = C::HPR, NH = WIDE ? 2 : 1;
    constexpr int QW = WIDE ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, kq = lane & 3;

    Cursor<ST> ic = locate<ST>(a, b, x, lane);   // the next step to copy
    Cursor<ST> cc = ic;                          // the next step to compute

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
    // The next row's fragments are loaded when the copies reach it, so that
    // their latency passes beside the current row's last steps: tag counts rows.
    uint32_t qa[D / 16][QW], qn[D / 16][QW];
    int copy_row = 0, row_no = 0, tag = 0;
    load_q(qn, ic);

    const uint32_t ring = smem_addr(gring);
    int issued = 0;
    // Block-table windows of 32 entries, in the lanes (a step's blocks, at most
    // 8 and aligned to their number, never straddle one): the current one, the
    // one after it, the sequence's first and the next sequence's first.
    int tab_s = -1, win = 0, tab = 0, tab_after = 0, tab_first = 0, win_first = 0;
    int seq_s = -1, seq_tab = 0;
    auto entries = [&](int s, const Seq& q, int from) -> int {
        const int i = from + lane;
        return i <= (q.n - 1) >> a.lgB ? a.tables[(int64_t)s * a.max_blocks + i] : -1;
    };
    auto first_window = [&](const Seq& q) { return (q.lo >> a.lgB) & ~7; };
    // Copy the step at ic into stage `st`: boxes of tpc tokens, those with a
    // visible one.
    auto issue = [&](int st) {
        const int t0 = (ic.q.j0 + ic.j) * ST;
        const int t1 = min(t0 + ST, ic.q.n);
        int tok = max(t0, ic.q.lo) & -a.tpc;
        const int first = tok >> a.lgB;
        if (ic.s != tab_s) {                        // another sequence
            win_first = first_window(ic.q);
            tab_first = seq_s == ic.s ? seq_tab : entries(ic.s, ic.q, win_first);
            tab_s = ic.s;
            win = -32;
            // look up the one after it
            seq_s = ic.s;
            Seq q;
            do {
                ++seq_s;
                q = seq_of<ST>(a, seq_s < a.S ? b.ctx[seq_s] : 1);
            } while (q.steps == 0);
            if (seq_s < a.S) seq_tab = entries(seq_s, q, first_window(q));
        }
        if ((unsigned)(first - win) >= 32u) {
            if (first == win + 32 && win >= 0) {
                win = first;
                tab = tab_after;
            } else if ((unsigned)(first - win_first) < 32u) {
                win = win_first;
                tab = tab_first;
            } else {
                win = first & ~7;
                tab = entries(ic.s, ic.q, win);
            }
            tab_after = entries(ic.s, ic.q, win + 32);
        }
        if (lane == 0)
            mbar_arrive_expect_tx(full + st, (uint32_t)((t1 - tok + a.tpc - 1) & -a.tpc) *
                                                 (uint32_t)(4 * D));
        for (; tok < t1; tok += a.tpc) {
            int phys = __shfl_sync(kFull, tab, (tok >> a.lgB) - win);
            if (lane == 0) {
                if ((unsigned)phys >= (unsigned)a.num_blocks) {
                    atomicOr(a.err, PKV_DEVERR_BAD_BLOCK);
                    phys = 0;                               // a valid row; flagged
                }
                const int y = ((phys * a.HK + ic.hk) << a.lgB) + (tok & ((1 << a.lgB) - 1));
                const uint32_t dst = ring + st * C::STAGE + (tok - t0) * (2 * D);
                tensor_g2s3(dst, &tk, 0, 0, y, full + st);
                tensor_g2s3(dst + C::HALF, &tv, 0, 0, y, full + st);
            }
        }
        ++issued;
        if (ic.next(a, b)) {
            ++copy_row;
            if (!WIDE && issued < left && tag <= row_no) {
                load_q(qn, ic);
                tag = copy_row;
            }
        }
    };

    for (int i = 0; i < kStages && issued < left; ++i) issue(i);

    float m[NH], l[NH], slope[NH];
    float acc[D / 8][4];
    bool began_before = cc.j > 0;
    int heads = 0;
    bool fresh = true, ok = true;

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
    for (int done = 0; done < left; ++done) {
        if (fresh) {
            fresh = false;
            if (tag == row_no) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int e = 0; e < QW; ++e) qa[kk][e] = qn[kk][e];
            } else {
                load_q(qa, cc);
            }
            heads = min(HPR, a.G - cc.gc * HPR);
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
        }
        if (!wait_phase(full + st, phase, nullptr, a.wait_ns)) {
            ok = false;
            break;
        }
        const int t0 = (cc.q.j0 + cc.j) * ST;
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
        if (a.cap_log2 > 0.f)               // cap tanh(y) = cap (1 - 2 / (2^(2 log2(e) y) + 1))
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
            const bool up = mx[i] > m[i] + kRaiseLog2 || m[i] == -INFINITY;
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
        each([&](float& y, int, int i) { y = ex2(y - m[i]); });
        if (edge)                           // (m is -infinity where every visible score is)
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
        // the stage is free: its values are in registers (and a zeroed row is
        // written before the next copy lands over it)
        if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (issued < left) issue(st);
        if (++st == kStages) {
            st = 0;
            phase ^= 1u;
        }

        const bool row_end = cc.j + 1 == cc.q.steps;
        if (row_end || done + 1 == left) {
            // the row's part in this range ends here
            const bool whole = row_end && !began_before;
            // (a row that goes on is the warp's last: every copy has landed and
            // been read, so its part may take the ring's place)
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
                p.last = (int)cut.run_of(x + done + (cc.q.steps - 1 - cc.j));
                meta[began_before ? 0 : 1] = p;
            }
            began_before = false;
            fresh = true;
        }
        if (cc.next(a, b)) ++row_no;
    }
    if (!ok) {
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        // let every copy issued land before the CTA can end
        for (int g = issued - kStages < 0 ? 0 : issued - kStages; g < issued; ++g)
            wait_phase(full + g % kStages, (uint32_t)((g / kStages) & 1), nullptr, kWaitLimitNs);
    }
}

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
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
    int* sums = reinterpret_cast<int*>(parts + 2 * kWarps);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = (int)blockIdx.x;
    uint64_t* full = bars + warp * kStages;
    if (tid == 0) {
        prefetch_map(&tk);
        prefetch_map(&tv);
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    if (lane < 2) parts[2 * warp + lane].s = -1;
    grid_dependency_wait();

    // steps before each thread's sequences
    Batch b;
    b.per = (a.S + kThreads - 1) / kThreads;
    b.prefix = prefix;
    b.ctx = b.per > 1 ? a.ctx : ctx;
    {
        int local = 0;
        for (int s = tid * b.per; s < a.S && s < (tid + 1) * b.per; ++s) {
            const int n = a.ctx[s];
            if (b.per == 1) ctx[tid] = n;
            local += seq_of<ST>(a, n).steps;
            if ((n < 0 || n > a.cap_tokens) && c == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
        }
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            if (i < warp) incl += sums[i];
        prefix[tid + 1] = incl;
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
    }
    grid_launch_dependents();

    // this CTA's run of the steps, this warp's run of it
    const int64_t X = (int64_t)(a.HK * a.chunks) * prefix[kThreads];
    const int64_t most = X / kMinSteps > 1 ? X / kMinSteps : 1;
    const int64_t used = X == 0 ? 0 : most < a.ctas ? most : a.ctas;
    bool recorded = false;
    if (c < used) {
        const Cut cut(X, used);
        const int64_t cx = cut.begin(c);
        const int cn = (int)(cut.begin(c + 1) - cx);
        const int each = cn / kWarps, longer = cn - each * kWarps;
        const int64_t x = cx + warp * each + min(warp, longer);
        const int left = each + (warp < longer);
        unsigned char* gring = base + warp * C::RING;
        if (left > 0)
            walk<T, D, WIDE>(tk, tv, a, b, x, left, gring, base + C::PARTS_OFF + warp * C::PART,
                             full, parts + 2 * warp, cut);
        __syncthreads();

        // Join the parts of each row, a head of a row a warp: a row begins with
        // an odd part, or with the CTA's first where it began in an earlier CTA.
        constexpr int V = D / 32;
        int unit = 0;
        for (int i = 0; i < 2 * kWarps;) {
            if (parts[i].s < 0) {
                ++i;
                continue;
            }
            const int first = i;
            const Part row = parts[first];
            bool ended = false;
            unsigned set = 0;
            for (; i < 2 * kWarps && !ended; ++i)
                if (parts[i].s >= 0) {
                    set |= 1u << i;
                    ended = parts[i].ended != 0;
                }
            const bool begins = (first & 1) != 0;
            if (begins && !ended) {
                recorded = true;
                if (tid == 0) {
                    Record rec;
                    rec.s = row.s;
                    rec.row = row.row;
                    rec.last = row.last;
                    rec.pad = 0;
                    a.rec[c] = rec;
                }
            }
            const int hk = row.row / a.chunks, gc = row.row - hk * a.chunks;
            const int heads = min(HPR, a.G - gc * HPR);
            for (int h = (warp + kWarps - unit % kWarps) % kWarps; h < heads; h += kWarps) {
                float M = -INFINITY, L = 0.f, o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = 0.f;
                auto part = [&](int k) -> const unsigned char* {
                    return k & 1 ? base + (k >> 1) * C::RING : base + C::PARTS_OFF + (k >> 1) * C::PART;
                };
                for (unsigned left_set = set; left_set; left_set &= left_set - 1)
                    M = fmaxf(M, reinterpret_cast<const float2*>(part(__ffs(left_set) - 1) +
                                                                 HPR * D * 4)[h].x);
                for (unsigned left_set = set; left_set; left_set &= left_set - 1) {
                    const unsigned char* p = part(__ffs(left_set) - 1);
                    const float2 ml = reinterpret_cast<const float2*>(p + HPR * D * 4)[h];
                    const float* v = reinterpret_cast<const float*>(p) + h * D + lane * V;
                    const float f = ex2(ml.x - M);
                    L += f * ml.y;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += f * v[e];
                }
                if (begins && ended) {
                    const float inv = 1.f / L;
                    uint32_t* out = reinterpret_cast<uint32_t*>(a.out) +
                                    ((int64_t)row.s * a.H + hk * a.G + gc * HPR + h) * (D / 2) +
                                    lane * (V / 2);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e)
                        out[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
                } else {
                    const int64_t to = (2 * (int64_t)c + (begins ? 1 : 0)) * HPR + h;
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
        for (int64_t i = tid; i < row_words; i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
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
    cfg.blockDim = dim3(kThreads);
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
    if ((int64_t)max_blocks * B >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: context capacity overflows", fn);
    const int st = kStepTokens * 128 / D;
    const int64_t steps = (int64_t)S * (((int64_t)max_blocks * B + st - 1) / st);
    if (steps >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: batch too large (step count overflows)", fn);
    out->G = H / HK;
    out->heads = out->G <= 8 ? 8 : 16;
    out->chunks = (out->G + out->heads - 1) / out->heads;
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

    const double log2e = 1.4426950408889634;
    char* ws = static_cast<char*>(workspace);
    Args a;
    a.out = out;
    a.q = q;
    a.tables = block_tables;
    a.ctx = context_lens;
    a.slopes = slopes;
    a.score = (float)(softcap > 0.f ? 2.0 * log2e * scale / softcap : log2e * scale);
    a.cap_log2 = (float)(log2e * softcap);
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
