// C ABI of the prompt phase with shared key/value heads, capped scores, a
// sliding window and a distance bias: argument checks, tensor maps, dispatch to
// the kind of kernel the arguments ask for.
#include <cmath>

#include "prefill_kernel.cuh"

namespace {

// Heads of a query tile: of the divisors of a K/V head's G that leave at least
// nine tenths of the tile's 128 rows used (where none does, of the one that uses
// most), the largest whose items are few enough to be dealt quickly, else the
// smallest above 1.  More heads a tile read the cache once for more of them and
// fill it with fewer tokens (8 sequences of 4 new tokens, 6000 cached, G = 8: 237
// -> 87 us against two heads an item), but a batch of many short items spends
// more on its schedule (40 prompts of 800, G = 16: 322 us with 16, 239 with 2).
int heads_of_tile(int G, int S, int max_query_len) {
    int best = 1, used = 0, few = 0;
    for (int gb = G < kBM ? G : kBM; gb >= 1; --gb) {
        if (G % gb != 0) continue;
        const int tb = kBM / gb, rows = tb * gb;
        if (10 * rows >= 9 * kBM) {
            const int64_t items = S * (((int64_t)max_query_len + 2 * tb - 1) / (2 * tb));
            if (items <= kDealItems / 2) return gb;
            if (gb > 1 || few == 0) few = gb;
        }
        if (rows > used) {
            used = rows;
            best = gb;
        }
    }
    return few ? few : best;
}

// Most work of CTAs: the items (of `tiles` query tiles) of max_query_len new tokens
// by groups of heads.
int64_t most_work(int S, int H, int gb, int max_query_len, int tiles) {
    const int tokens = tiles * (kBM / gb);
    return (int64_t)S * (((int64_t)max_query_len + tokens - 1) / tokens) * (H / gb);
}

// Whether a batch of these sizes may have so few units that its items are cut
// along the keys.  The lengths are on the device: this goes by upper bounds of the
// work (items by groups of heads) and of an item's key tiles.  A batch that turns
// out not to be cut pays for the second launch and the estimate (about 5 us), so
// work for half of the SMs or less asks for 8 tiles, for all of them 16 (4 prompts
// of 2-194 over 3798, 40/8 heads x 64: 92 -> 63 us; 2 of 512 over 4000, which are
// not cut: 91 -> 96).  The capacity is the table's, so short prompts in a server's
// wide table pay it too (one of 61 tokens, 32/8 x 128: 9.3 us in a table of under
// 1024 tokens or without a workspace, 13.6 with one): their callers give none.
bool may_split(int S, int H, int HK, int B, int max_blocks, int max_query_len, int window) {
    const int gb = heads_of_tile(H / HK, S, max_query_len);
    int64_t keys = (int64_t)max_blocks * B;
    if (window > 0 && keys > (int64_t)window + 2 * (kBM / gb)) keys = window + 2 * (kBM / gb);
    const int64_t work = most_work(S, H, gb, max_query_len, 2);
    return S <= kSplitItems && (work <= kSplitParts / 4 ? keys >= 8 * kBN
                                                       : work <= kSplitParts / 2 && keys >= 16 * kBN);
}

struct SplitLayout {
    size_t units, ml, acc, total;
};
SplitLayout split_layout(int D) {
    SplitLayout l;
    const size_t rows = (size_t)kSplitParts * 2 * kBM;
    l.units = pkv::align_up(sizeof(SplitHead), 256);
    l.ml = pkv::align_up(l.units + sizeof(SplitUnit) * kSplitParts, 256);
    l.acc = l.ml + 8 * rows;
    l.total = l.acc + 4 * rows * (size_t)D;
    return l;
}

}  // namespace

extern "C" {

pkv_status pkv_prefill_grouped_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                              int head_dim, int block_size, int max_blocks_per_seq,
                                              int max_query_len, size_t* bytes) {
    const char* fn = "pkv_prefill_grouped_workspace_size";
    if (!bytes) return pkv::fail(PKV_ERR_INVALID, "%s: bytes is NULL", fn);
    if (num_seqs < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128) || block_size < 1 || max_blocks_per_seq < 1 ||
        max_query_len < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    *bytes = may_split(num_seqs, num_heads, num_kv_heads, block_size, max_blocks_per_seq,
                       max_query_len, 0)
                 ? split_layout(head_dim).total : 0;
    return PKV_OK;
}

pkv_status pkv_paged_attention_prefill_grouped(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
    const float* slopes, float scale, float softcap, int window, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    int max_query_len, int num_query_tokens, pkv_dtype dtype, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
    const char* fn = "pkv_paged_attention_prefill_grouped";
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv::fail(PKV_ERR_INVALID, "%s: num_seqs must be in [0, 65535]", fn);
    if (num_heads < 1 || num_heads > 65535 || num_kv_heads < 1 || num_heads % num_kv_heads != 0)
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_heads must be a multiple of num_kv_heads, at most 65535", fn);
    if (head_dim != 64 && head_dim != 128)
        return pkv::fail(PKV_ERR_INVALID, "%s: head_dim must be 64 or 128", fn);
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        return pkv::fail(PKV_ERR_INVALID, "%s: block_size must be 8, 16, 32 or 64", fn);
    if (max_blocks_per_seq < 1 || max_query_len < 0 || num_query_tokens < 0)
        return pkv::fail(PKV_ERR_INVALID, "%s: bad sizes", fn);
    if ((int64_t)max_blocks_per_seq * block_size > (1LL << 30))
        return pkv::fail(PKV_ERR_INVALID, "%s: context capacity above 2^30 tokens", fn);
    // the tiled copies address cache rows (block, head, token) with 32-bit coordinates
    if (num_blocks < 1 || num_blocks > ((1LL << 31) - 1) / ((int64_t)num_kv_heads * block_size))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: num_blocks must be >= 1, and num_blocks * num_kv_heads * block_size "
                         "below 2^31",
                         fn);
    if (dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::fail(PKV_ERR_INVALID, "%s: unknown dtype", fn);
    const int gb = heads_of_tile(num_heads / num_kv_heads, num_seqs, max_query_len);
    {
        // the work schedule sums item costs in 64 bits: a bound far above any
        // call whose tensors fit in memory
        const double units =
            (double)most_work(num_seqs, num_heads, gb, max_query_len, 2);
        const double unit_cost =
            kPairCost * ((double)max_blocks_per_seq * block_size / kBN + 1.0) + kItemCost;
        if (units * unit_cost >= 0x1p60)
            return pkv::fail(PKV_ERR_INVALID, "%s: too much work for one call", fn);
    }
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
    if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start)
        return pkv::fail(PKV_ERR_INVALID, "%s: NULL pointer", fn);
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return pkv::fail(PKV_ERR_INVALID, "%s: out, q and the caches must be 16-byte aligned", fn);
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) ||
        !aligned(slopes, 4))
        return pkv::fail(PKV_ERR_INVALID,
                         "%s: block_tables, context_lens, query_start and slopes must be 4-byte "
                         "aligned",
                         fn);
    const bool split = workspace && may_split(num_seqs, num_heads, num_kv_heads, block_size,
                                              max_blocks_per_seq, max_query_len, window);
    const SplitLayout lay = split_layout(head_dim);
    if (split && !aligned(workspace, 256))
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace must be 256-byte aligned", fn);
    if (split && workspace_bytes < lay.total)
        return pkv::fail(PKV_ERR_INVALID, "%s: workspace too small (%zu < %zu bytes)", fn,
                         workspace_bytes, lay.total);
    int32_t* err = pkv::device_error_word();
    if (!err) return pkv::fail(PKV_ERR_CUDA, "%s: no CUDA device", fn);

    const bool bf16 = dtype == PKV_BF16;
    CUtensorMap tq, tk, tv;
    {
        // q: [tokens][heads][D], one box = tb tokens x gb heads x 64 elements
        const cuuint64_t D = (cuuint64_t)head_dim;
        const cuuint64_t dims[3] = {D, (cuuint64_t)num_heads, (cuuint64_t)num_query_tokens};
        const cuuint64_t strides[2] = {D * 2, (cuuint64_t)num_heads * D * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)gb, (cuuint32_t)(kBM / gb)};
        if (!make_map(&tq, bf16, 3, q, dims, strides, box))
            return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of q", fn);
    }
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    if (!pkv::pool_map(&tk, bf16, k_cache, rows, head_dim, block_size) ||
        !pkv::pool_map(&tv, bf16, v_cache, rows, head_dim, block_size))
        return pkv::fail(PKV_ERR_CUDA, "%s: tensor map of the caches", fn);

    PrefillArgs a = {};
    a.out = out;
    a.out_v8 = aligned(out, 32) ? 1 : 0;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.scale_log2 = large_cap ? 1.f : score;
    a.S = num_seqs;
    a.H = num_heads;
    a.B = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.max_query_len = max_query_len;
    a.num_tokens = num_query_tokens;
    a.HK = num_kv_heads;
    a.G = num_heads / num_kv_heads;
    a.window = window;
    a.cap_log2 = cap_log2;
    a.cap_scale = scale;
    a.cap_inv = large_cap ? (float)(1.0 / softcap) : 0.f;
    a.slopes = slopes;
    const bool lifted =
        a.G > 1 || window > 0 || max_blocks_per_seq * block_size > kPlainTokens;
    a.lift = lifted ? kLift : 0.f;
    a.rescale = lifted ? kLiftRescale : kRescaleLog2;
    a.up = lifted ? kLiftUp : 0.f;
    a.gb = gb;
    a.tb = kBM / gb;
    a.head_units = num_heads / gb;
    a.units_per_kv = a.G / gb;
    a.per = a.head_units % 2 == 0 ? 2 : 1;
    // Items of one tile where every such item can have an SM of its own: the two of
    // an item would share one (one prompt, 32/8 heads x 128, bf16: of 61 tokens 9.85 ->
    // 9.1 us, of 125 11.4 -> 9.8).  Not in the cut kind, whose bounds count items of two.
    int dev = 0;
    const cudaError_t de = cudaGetDevice(&dev);
    if (de != cudaSuccess) return pkv::cuda_fail(de, fn);
    const bool one = !split && most_work(num_seqs, num_heads, gb, max_query_len, 1) <=
                                   pkv::sm_count(dev);
    a.item_tokens = one ? a.tb : 2 * a.tb;
    a.q_items = (int)(((int64_t)max_query_len + a.item_tokens - 1) / a.item_tokens);
    a.num_blocks = num_blocks;
    if (split) {
        a.most_work = (int)most_work(num_seqs, num_heads, gb, max_query_len, 2);
        char* ws = static_cast<char*>(workspace);
        a.split = reinterpret_cast<SplitHead*>(ws);
        a.split_units = reinterpret_cast<SplitUnit*>(ws + lay.units);
        a.split_ml = reinterpret_cast<float2*>(ws + lay.ml);
        a.split_acc = reinterpret_cast<float*>(ws + lay.acc);
    }
    a.err = err;
    const int kind = kGrouped | (softcap > 0.f && !large_cap ? kCapped : 0) |
                     (slopes || large_cap ? kBiased : 0);
    pkv::LaunchGrouped* const launch =
        split ? (bf16 ? pkv::launch_prefill_cut_bf16 : pkv::launch_prefill_cut_f16)
              : (bf16 ? pkv::launch_prefill_grouped_bf16 : pkv::launch_prefill_grouped_f16);
    const cudaError_t e = launch(tq, tk, tv, a, head_dim, kind, stream);
    if (e != cudaSuccess) return pkv::cuda_fail(e, fn);
    return PKV_OK;
}

}  // extern "C"
