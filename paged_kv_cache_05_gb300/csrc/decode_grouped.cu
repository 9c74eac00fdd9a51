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
// tensor-core products (register operands; their rate is far above what the
// memory can feed, so the fifth-generation unit has nothing to add here).
//
// Design.  The work is the ordered space of steps (s, row, j): a row is a K/V
// head and up to 8 (G <= 8) or 16 of its query heads, a step ST tokens (4 KiB
// of K and as much of V).  The space is cut into equal ranges, one per WARP of
// a persistent grid, whatever the mix of lengths: a warp shares nothing with
// the others of its block.  It walks its range with a ring of kStages stages
// of its own, into which its lanes issue tiled bulk copies (128-byte swizzle,
// so that ldmatrix meets no bank conflict) kStages steps ahead, one mbarrier
// a stage.
//   S = Q K^T: the heads are the product's 16 rows, the tokens its columns;
//   online softmax in log2 units, a row's statistics in the four lanes that
//   hold it; P goes straight from S's registers to the operand of O += P V.
//   P is split into a 16-bit high part and the 16-bit residual, so weights keep
//   at least 16 bits.  With up to 8 heads, rows 8-15 of the product are free:
//   the residual takes them, and O is the sum of row r and row r + 8 at the
//   end, at no further product.  With 9 to 16 heads the residual is a second
//   product.
// A range ends in at most two partial rows (running max, sum, unnormalised
// output): one that began in an earlier range and one that goes on in later
// ones.  The range in which a split row begins records it, and a second kernel
// joins its parts in range order, so results do not vary from call to call.
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

constexpr int kWarps = 4;                   // ranges per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;                  // ring stages per warp, 8 KiB each
constexpr int kCtasPerSm = 2;
constexpr int kMaxRanges = 2048;
constexpr int kMinSteps = 2;                // fewest steps of a range
constexpr float kRaiseLog2 = 8.f;           // raise the running max only past this growth

template <int D>
struct Geo {
    static constexpr int ST = pkv::step_tokens(D);      // 16 or 32 tokens
    static constexpr int SLABS = D / 64;                // 128-byte column slabs of a row
    static constexpr int HALF = ST * D * 2;             // bytes of a step's K (or V)
    static constexpr int STAGE = 2 * HALF;
    static constexpr int SUBS = ST / 16;
    static constexpr size_t RING = (size_t)kWarps * kStages * STAGE;
    static constexpr size_t SMEM = 1024 + RING + 8 * kWarps * kStages + 4 * (kThreads + 1);
};

// A split row, recorded by the range in which it begins.
struct Record {
    int s, row, last, pad;                  // s < 0: none; last: the range it ends in
};

struct Args {
    void* out;
    const void* q;
    const int32_t* tables;
    const int32_t* ctx;
    const float* slopes;
    float score;           // without a cap: scale * log2(e), else 2 log2(e) scale / cap
    float cap_log2;        // cap * log2(e); 0: no cap
    int window, S, H, HK, G, chunks, max_blocks, lgB, tpc;
    int ranges;            // warps of the grid
    int64_t num_blocks;
    uint64_t wait_ns;
    Record* rec;           // [ranges]
    float2* ml;            // [2 ranges][heads a row]: running max (log2), sum
    float* acc;            // [2 ranges][heads a row][D]
    int32_t* err;
};

// One sequence's tokens in steps.
struct Seq {
    int n, lo, j0, steps;
};
template <int ST>
__device__ __forceinline__ Seq seq_of(const Args& a, int s, bool* bad = nullptr) {
    Seq q;
    const int cap = (int)(((int64_t)a.max_blocks << a.lgB) < 0x7fffffff
                              ? ((int64_t)a.max_blocks << a.lgB) : 0x7fffffff);
    const int c = a.ctx[s];
    if (bad) *bad = c < 0 || c > cap;
    q.n = c < 0 ? 0 : c > cap ? cap : c;
    q.lo = a.window > 0 && q.n > a.window ? q.n - a.window : 0;
    q.j0 = q.lo / ST;
    q.steps = q.n > 0 ? (q.n - 1) / ST + 1 - q.j0 : 0;
    return q;
}

// A place in the step space: step j (from 0) of row `row` of sequence s.
template <int ST>
struct Cursor {
    int s, row, j;
    Seq q;
    __device__ __forceinline__ void next(const Args& a, int rows) {
        if (++j < q.steps) return;
        j = 0;
        if (++row < rows) return;
        row = 0;
        do {
            ++s;
            if (s >= a.S) return;
            q = seq_of<ST>(a, s);
        } while (q.steps == 0);
    }
};

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    grouped_decode_main(const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const Args a) {
    using C = Geo<D>;
    constexpr int ST = C::ST, SUBS = C::SUBS, HPR = WIDE ? 16 : 8;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + C::RING);
    int* prefix = reinterpret_cast<int*>(bars + kWarps * kStages);   // [kThreads + 1]
    __shared__ int warp_sum_[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, kq = lane & 3;
    uint64_t* full = bars + warp * kStages;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    grid_dependency_wait();

    // steps before each thread's sequences
    const int per = (a.S + kThreads - 1) / kThreads;
    {
        int local = 0;
        for (int s = tid * per; s < a.S && s < (tid + 1) * per; ++s) {
            bool bad;
            local += seq_of<ST>(a, s, &bad).steps;
            if (bad && blockIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_CONTEXT);
        }
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum_[warp] = incl;
        __syncthreads();
        for (int i = 0; i < warp; ++i) incl += warp_sum_[i];
        prefix[tid + 1] = incl;
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
    }
    grid_launch_dependents();

    // rows that attend nothing
    const int64_t row_words = (int64_t)a.H * D / 8;
    for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
        if (a.ctx[s] > 0) continue;
        uint4* o = static_cast<uint4*>(a.out) + s * row_words;
        for (int64_t i = tid; i < row_words; i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }

    // this warp's range [x, x1) of the steps
    const int rows = a.HK * a.chunks;
    const int64_t X = (int64_t)rows * prefix[kThreads];
    const int64_t most = X / kMinSteps > 1 ? X / kMinSteps : 1;
    const int64_t W = X == 0 ? 0 : most < a.ranges ? most : a.ranges;
    const int w = warp * (int)gridDim.x + (int)blockIdx.x;
    if (w >= W) {
        if (lane == 0) a.rec[w].s = -1;
        return;
    }
    int64_t x = w * X / W;
    const int left_all = (int)((w + 1) * X / W - x);

    Cursor<ST> ic;                          // the next step to copy
    {
        int lo = 0, hi = kThreads - 1;      // the thread whose sequences hold x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)rows * prefix[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        int64_t before = prefix[lo];
        const int end = min(a.S, (lo + 1) * per);
        ic.s = -1;
        for (int s0 = lo * per; s0 < end; s0 += 32) {
            const int s = s0 + lane;
            int n = s < end ? seq_of<ST>(a, s).steps : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned hit = __ballot_sync(kFull, (before + incl) * rows > x);
            if (hit) {
                const int f = __ffs(hit) - 1;
                ic.s = s0 + f;
                before += __shfl_sync(kFull, incl - n, f);
                break;
            }
            before += __shfl_sync(kFull, incl, 31);
        }
        ic.q = seq_of<ST>(a, ic.s);
        const int64_t in = x - before * rows;
        ic.row = (int)(in / ic.q.steps);
        ic.j = (int)(in - (int64_t)ic.row * ic.q.steps);
    }
    Cursor<ST> cc = ic;                     // the next step to compute

    const uint32_t ring = base + warp * (kStages * C::STAGE);
    unsigned char* gring = gbase + warp * (kStages * C::STAGE);
    int issued = 0;
    int tab_s = -1, win = 0, tab = 0, tab_next = 0;
    auto entries = [&](const Cursor<ST>& c, int first) -> int {
        const int i = first + lane;
        return i <= (c.q.n - 1) >> a.lgB ? a.tables[(int64_t)c.s * a.max_blocks + i] : -1;
    };
    // Copy the step at ic into stage `st`: boxes of tpc tokens x 64 columns.
    auto issue = [&](int st) {
        const int t0 = (ic.q.j0 + ic.j) * ST;
        const int first = max(t0, ic.q.lo) >> a.lgB;
        const int last = (min(t0 + ST, ic.q.n) - 1) >> a.lgB;
        if (ic.s != tab_s || first < win || last >= win + 32) {
            if (ic.s == tab_s && (first & ~3) == win + 32) {
                win += 32;
                tab = tab_next;
            } else {
                win = first & ~3;
                tab = entries(ic, win);
                tab_s = ic.s;
            }
            tab_next = entries(ic, win + 32);
        }
        const int boxes = ST / a.tpc;                       // per 64 columns
        const int box = lane >> C::SLABS;                   // lane = (box, slab, K or V)
        const int slab = C::SLABS == 2 ? (lane >> 1) & 1 : 0;
        const int tok = t0 + box * a.tpc;
        const bool on = box < boxes && tok < ic.q.n && tok + a.tpc > ic.q.lo;
        int64_t phys = __shfl_sync(kFull, tab, ((tok >> a.lgB) - win) & 31);
        const unsigned all = __ballot_sync(kFull, on);
        if (lane == 0)
            mbar_arrive_expect_tx(full + st, (uint32_t)(__popc(all) * a.tpc * 128));
        __syncwarp();
        if (on) {
            if (phys < 0 || phys >= a.num_blocks) {
                atomicOr(a.err, PKV_DEVERR_BAD_BLOCK);
                phys = 0;                                   // a valid row; flagged
            }
            const int y = (int)(((phys * a.HK + ic.row / a.chunks) << a.lgB) +
                                (tok & ((1 << a.lgB) - 1)));
            unsigned char* dst = gring + st * C::STAGE + (lane & 1) * C::HALF +
                                 slab * (ST * 128) + box * a.tpc * 128;
            tensor_g2s(dst, lane & 1 ? &tv : &tk, slab * 64, y, full + st);
        }
        ++issued;
        ic.next(a, rows);
    };

    for (int i = 0; i < kStages && issued < left_all; ++i) issue(i);

    uint32_t qa[D / 16][WIDE ? 4 : 2];
    float m[WIDE ? 2 : 1], l[WIDE ? 2 : 1], slope[WIDE ? 2 : 1];
    float acc[D / 8][4];
    bool began_before = cc.j > 0;
    int heads = 0, head0 = 0;
    bool fresh = true, ok = true;
    bool recorded = false;

    // fragment rows of this lane in the swizzled tiles
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t krow = (uint32_t)(((mi >> 1) * 8 + mr) * 128);     // K: token, chunk parity mi & 1
    const uint32_t vrow = (uint32_t)(((mi & 1) * 8 + mr) * 128);      // V: token, chunk parity mi >> 1

    for (int done = 0; done < left_all; ++done) {
        const int st = done % kStages;
        if (fresh) {
            fresh = false;
            const int gc = cc.row % a.chunks;
            heads = min(HPR, a.G - gc * HPR);
            head0 = (cc.row / a.chunks) * a.G + gc * HPR;
            const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q) +
                                 ((int64_t)cc.s * a.H + head0 + r) * (D / 2) + kq;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][0] = r < heads ? qr[kk * 8] : 0u;
                qa[kk][1] = r < heads ? qr[kk * 8 + 4] : 0u;
                if constexpr (WIDE) {
                    qa[kk][2] = r + 8 < heads ? qr[kk * 8 + 8 * (D / 2)] : 0u;
                    qa[kk][3] = r + 8 < heads ? qr[kk * 8 + 4 + 8 * (D / 2)] : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
                slope[i] = a.slopes && r + 8 * i < heads
                               ? a.slopes[head0 + r + 8 * i] * 1.4426950408889634f : 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        }
        if (!wait_phase(full + st, (uint32_t)((done / kStages) & 1), nullptr, a.wait_ns)) {
            ok = false;
            break;
        }
        const int t0 = (cc.q.j0 + cc.j) * ST;
        const bool edge = t0 < cc.q.lo || t0 + ST > cc.q.n;
        const uint32_t sk = ring + st * C::STAGE, sv = sk + C::HALF;
        if (edge) {
            for (int i = lane; i < ST * C::SLABS * 8; i += 32) {
                const int tok = (i >> 3) % ST;
                if (t0 + tok < cc.q.lo || t0 + tok >= cc.q.n)
                    *reinterpret_cast<uint4*>(gring + st * C::STAGE + C::HALF + i * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
        }

        float z[SUBS][2][4];
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[u][0][e] = z[u][1][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kb[4];
                const int chunk = (2 * kk + (mi & 1)) & 7;
                ldsm_x4(kb, sk + (kk >> 2) * (ST * 128) + u * 2048 + krow + ((chunk ^ mr) << 4));
                const uint32_t af[4] = {qa[kk][0], WIDE ? qa[kk][WIDE ? 2 : 0] : 0u, qa[kk][1],
                                        WIDE ? qa[kk][WIDE ? 3 : 0] : 0u};
                mma16816<T>(z[u][0], af, kb[0], kb[1]);
                mma16816<T>(z[u][1], af, kb[2], kb[3]);
            }
        }

        float alpha[WIDE ? 2 : 1];
        bool raised = false;
#pragma unroll
        for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& s = z[u][v][2 * i + e];
                        const int t = t0 + u * 16 + v * 8 + 2 * kq + e;
                        s *= a.score;
                        // cap tanh(y) = cap (1 - 2 / (2^(2 log2(e) y) + 1))
                        if (a.cap_log2 > 0.f)
                            s = a.cap_log2 * (1.f - __fdividef(2.f, exp2f(s) + 1.f));
                        if (a.slopes) s += slope[i] * (float)(t - (cc.q.n - 1));
                        if (edge && (t < cc.q.lo || t >= cc.q.n)) s = -INFINITY;
                        mx = fmaxf(mx, s);
                    }
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const bool up = mx > m[i] + kRaiseLog2 || m[i] == -INFINITY;
            alpha[i] = up ? exp2f(m[i] - mx) : 1.f;
            if (up) m[i] = mx;
            raised |= up;
        }
        if (__any_sync(kFull, raised)) {
#pragma unroll
            for (int i = 0; i < (WIDE ? 2 : 1); ++i) l[i] *= alpha[i];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                acc[i][0] *= alpha[0];
                acc[i][1] *= alpha[0];
                acc[i][2] *= alpha[WIDE ? 1 : 0];
                acc[i][3] *= alpha[WIDE ? 1 : 0];
            }
        }
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
            uint32_t hi[2][WIDE ? 2 : 1], lo[2][WIDE ? 2 : 1];
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = t0 + u * 16 + v * 8 + 2 * kq + e;
                        p[e] = exp2f(z[u][v][2 * i + e] - m[i]);
                        if (edge && (t < cc.q.lo || t >= cc.q.n)) p[e] = 0.f;
                    }
                    l[i] += p[0] + p[1];
                    hi[v][i] = pack2<T>(p[0], p[1]);
                    const float2 h = unpack2<T>(hi[v][i]);
                    lo[v][i] = pack2<T>(p[0] - h.x, p[1] - h.y);
                }
            const uint32_t pa[4] = {hi[0][0], WIDE ? hi[0][WIDE ? 1 : 0] : lo[0][0], hi[1][0],
                                    WIDE ? hi[1][WIDE ? 1 : 0] : lo[1][0]};
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint32_t vb[4];
                const int chunk = (2 * c + (mi >> 1)) & 7;
                ldsm_x4_t(vb, sv + (c >> 2) * (ST * 128) + u * 2048 + vrow + ((chunk ^ mr) << 4));
                mma16816<T>(acc[2 * c], pa, vb[0], vb[1]);
                mma16816<T>(acc[2 * c + 1], pa, vb[2], vb[3]);
                if constexpr (WIDE) {
                    const uint32_t pl[4] = {lo[0][0], lo[0][1], lo[1][0], lo[1][1]};
                    mma16816<T>(acc[2 * c], pl, vb[0], vb[1]);
                    mma16816<T>(acc[2 * c + 1], pl, vb[2], vb[3]);
                }
            }
        }
        // the stage is free: its values are in registers (a zeroed row before
        // the next copy lands over it)
        if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        const bool row_end = cc.j + 1 == cc.q.steps;
        if (issued < left_all) issue(st);

        if (row_end || done + 1 == left_all) {
            // the row's part in this range ends here
            const bool whole = row_end && !began_before;
            const int slot = 2 * w + (began_before ? 0 : 1);
#pragma unroll
            for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
                float sum = l[i];
                sum += __shfl_xor_sync(kFull, sum, 1);
                sum += __shfl_xor_sync(kFull, sum, 2);
                const int hr = r + 8 * i;
                if (hr >= heads) continue;
                const float inv = 1.f / sum;
                uint32_t* o = reinterpret_cast<uint32_t*>(a.out) +
                              ((int64_t)cc.s * a.H + head0 + hr) * (D / 2) + kq;
                float2* pacc = reinterpret_cast<float2*>(a.acc + ((int64_t)slot * HPR + hr) * D) + kq;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const float o0 = WIDE ? acc[c][2 * i] : acc[c][0] + acc[c][2];
                    const float o1 = WIDE ? acc[c][2 * i + 1] : acc[c][1] + acc[c][3];
                    if (whole) o[c * 4] = pack2<T>(o0 * inv, o1 * inv);
                    else pacc[c * 4] = make_float2(o0, o1);
                }
                if (!whole && kq == 0) a.ml[(int64_t)slot * HPR + hr] = make_float2(m[i], sum);
            }
            if (!row_end && !began_before) {
                // the row begins here and goes on: find the range it ends in
                const int64_t at = x + done + (cc.q.steps - 1 - cc.j);
                if (lane == 0) {
                    Record rec;
                    rec.s = cc.s;
                    rec.row = cc.row;
                    rec.last = (int)(((at + 1) * W - 1) / X);
                    rec.pad = 0;
                    a.rec[w] = rec;
                }
                recorded = true;
            }
            began_before = false;
            fresh = true;
        }
        cc.next(a, rows);
    }
    if (!recorded && lane == 0) a.rec[w].s = -1;
    if (!ok) {
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        // let every copy issued land before the CTA can end
        for (int g = issued - kStages < 0 ? 0 : issued - kStages; g < issued; ++g)
            wait_phase(full + g % kStages, (uint32_t)((g / kStages) & 1), nullptr, kWaitLimitNs);
    }
}

// Joins the parts of each split row: with M the largest running max,
//   out = sum_k 2^(m_k - M) acc_k / sum_k 2^(m_k - M) l_k.
// One CTA per recorded row, a warp per head.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(128) grouped_decode_merge(const Args a) {
    constexpr int HPR = WIDE ? 16 : 8, V = D / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int w0 = blockIdx.x;
    const Record rec = a.rec[w0];
    if (rec.s < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gc = rec.row % a.chunks;
    const int heads = min(HPR, a.G - gc * HPR);
    const int head0 = (rec.row / a.chunks) * a.G + gc * HPR;
    const int parts = rec.last - w0 + 1;
    auto slot = [&](int k) -> int64_t { return 2 * (int64_t)(w0 + k) + (k == 0 ? 1 : 0); };
    for (int h = warp; h < heads; h += 4) {
        float M = -INFINITY;
        for (int k = lane; k < parts; k += 32) M = fmaxf(M, a.ml[slot(k) * HPR + h].x);
        M = warp_max(M);
        float o[V], L = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const float2 ml = a.ml[slot(k) * HPR + h];
            const float* p = a.acc + (slot(k) * HPR + h) * D + lane * V;
            const float f = exp2f(ml.x - M);
            L += f * ml.y;
            if constexpr (V == 4) {
                const float4 v = *reinterpret_cast<const float4*>(p);
                o[0] += f * v.x;
                o[1] += f * v.y;
                o[2] += f * v.z;
                o[3] += f * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(p);
                o[0] += f * v.x;
                o[1] += f * v.y;
            }
        }
        const float inv = 1.f / L;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out) +
                        ((int64_t)rec.s * a.H + head0 + h) * (D / 2) + lane * (V / 2);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) out[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
    }
}

template <typename T, int D, bool WIDE>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Args& a, int grid,
                   cudaStream_t stream) {
    const size_t smem = Geo<D>::SMEM;
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
    cfg.gridDim = dim3((unsigned)a.ranges);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, grouped_decode_merge<T, D, WIDE>, a);
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
// follow: query heads a row, rows per sequence, the most ranges.
struct Shape {
    int G, heads, chunks, ranges;
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
    const int64_t steps = (int64_t)S * pkv::max_steps_per_seq(D, B, max_blocks);
    if (steps >= (1LL << 31))
        return pkv::fail(PKV_ERR_INVALID, "%s: batch too large (step count overflows)", fn);
    out->G = H / HK;
    out->heads = out->G <= 8 ? 8 : 16;
    out->chunks = (out->G + out->heads - 1) / out->heads;
    // a CTA per range at most, so that few ranges spread over the SMs
    int64_t most = steps * HK * out->chunks / kMinSteps;
    most = most < 1 ? 1 : most < kMaxRanges / kWarps ? most : kMaxRanges / kWarps;
    out->ranges = (int)most * kWarps;
    return PKV_OK;
}

struct Layout {
    size_t ml, acc, total;
};
Layout layout_of(const Shape& s, int D) {
    Layout l;
    const size_t rows = 2 * (size_t)s.ranges * s.heads;
    l.ml = pkv::align_up(sizeof(Record) * (size_t)s.ranges, 256);
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
    // one wave, no more warps than ranges the batch could have
    int grid = sms * kCtasPerSm;
    if (grid > sh.ranges / kWarps) grid = sh.ranges / kWarps;

    CUtensorMap tk, tv;
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    const int box = block_size < 16 ? block_size : 16;
    if (!pkv::pool_map(&tk, dtype == PKV_BF16, k_cache, rows, head_dim, box) ||
        !pkv::pool_map(&tv, dtype == PKV_BF16, v_cache, rows, head_dim, box))
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
    a.lgB = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    a.tpc = box;
    a.ranges = grid * kWarps;
    a.num_blocks = num_blocks;
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
