// prefill.cu -- the pkv_paged_attention_prefill entry point (chunked prefill
// attention over the paged cache): argument checks, the row-tile and KV-split
// plan, and the launches of the persistent paged_prefill_tc_kernel and its
// merge.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "prefill_launch.cuh"

namespace {

constexpr int kMinSplitTokens = 512;  // a KV split covers at least 4 tiles

struct PrefillShape {
    int tile_tokens = 0;   // chunk tokens per row tile: 128 / group
    int row_tiles = 0;     // row tiles of the longest chunk
    int splits = 0;
    int split_tokens = 0;  // multiple of 128
    int items = 0;         // row_tiles * num_kv_heads * num_seqs * splits
};

pkv_status plan_prefill(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                        int block_size, int max_query_len, int max_context_len, int kv_splits,
                        int sm_count, PrefillShape *pp, int window = 0, bool has_prefix = false, int sinks = 0) {
    if (head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        max_query_len < 0 || max_context_len < max_query_len || kv_splits < 0 || sm_count <= 0 ||
        num_kv_heads > 65535)
        return PKV_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads;
    if (group > 128) return PKV_ERR_UNSUPPORTED;  // a row tile holds at least one token
    pp->tile_tokens = 128 / group;
    const int64_t row_tiles = (static_cast<int64_t>(max_query_len) + pp->tile_tokens - 1) / pp->tile_tokens;
    pp->row_tiles = static_cast<int>(row_tiles);
    // the longest token range of a row tile: with a window (and no prefix behind it) its
    // rows' windows, from the block that holds the first, behind the blocks of the first tokens
    if (window > 0 && !has_prefix)
        max_context_len = static_cast<int>(std::min<int64_t>(
            max_context_len, static_cast<int64_t>(window) + pp->tile_tokens - 1 + block_size - 1 +
                                 (static_cast<int64_t>(sinks) + block_size - 1) / block_size * block_size));
    const int64_t ctx_tiles = std::max<int64_t>(1, (max_context_len + 127) / 128);
    int64_t want = kv_splits;
    if (want == 0) {
        // split the KV range only when the row tiles alone leave SMs idle
        const int64_t units = std::max<int64_t>(1, row_tiles * num_kv_heads * num_seqs);
        want = units >= sm_count ? 1 : (sm_count + units - 1) / units;
        want = std::min<int64_t>(want, std::max<int64_t>(1, max_context_len / kMinSplitTokens));
    }
    want = std::min<int64_t>(want, ctx_tiles);
    const int64_t tiles_per_split = (ctx_tiles + want - 1) / want;
    pp->split_tokens = static_cast<int>(tiles_per_split * 128);
    pp->splits = static_cast<int>((ctx_tiles + tiles_per_split - 1) / tiles_per_split);
    if (static_cast<int64_t>(num_seqs) * pp->splits > 65535) return PKV_ERR_INVALID_ARG;
    const int64_t items = row_tiles * num_kv_heads * num_seqs * pp->splits;  // < 2^63
    if (items > 0x7fffffff) return PKV_ERR_INVALID_ARG;
    pp->items = static_cast<int>(items);
    return PKV_OK;
}

// The scored prefill plans its items on the device (paged_prefill_plan_kernel) when the
// KV ranges are not split and the row tiles fit the plan's one block.
bool planned(const PrefillShape &pp, int num_seqs) {
    return pp.splits == 1 && static_cast<int64_t>(pp.row_tiles) * num_seqs <= pkv::kMaxPlanEntries;
}

size_t prefill_workspace(int num_rows, int num_q_heads, int splits) {
    if (splits <= 1) return 0;
    return static_cast<size_t>(num_rows) * num_q_heads * splits * (128 + 2) * sizeof(float);
}

size_t plan_bytes(const PrefillShape &pp, int num_seqs) {
    return offsetof(pkv::PrefillPlan, entry) + sizeof(pkv::PrefillEntry) * static_cast<size_t>(pp.row_tiles) * num_seqs;
}

// What the scored prefill adds to a call.
struct ScoredPrefillArgs {
    float softcap;
    const float *slopes;
    int window;
    const int32_t *starts;
    const int32_t *prefix_lens;
    bool sink_form = false;  // a window and first tokens, nothing else
    int sinks = 0;
};

pkv_status prefill_impl(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, void *out, void *workspace, size_t workspace_bytes,
    int kv_splits, pkv_dtype dtype, void *stream, const ScoredPrefillArgs *scored) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads || num_blocks <= 0 || num_blocks > 0x7fffffffLL ||
        max_blocks_per_seq <= 0 || max_query_len < 0 || max_context_len < max_query_len ||
        static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size ||
        kv_splits < 0 || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    const int64_t half_elems = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_elems < half_elems || block_stride_elems % 8) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return PKV_ERR_INVALID_ARG;
    const int window = scored ? scored->window : 0;
    const bool has_prefix = scored && scored->prefix_lens;
    const bool sink_form = scored && scored->sink_form;
    const int sinks = scored ? scored->sinks : 0;
    if (sink_form && (window < 1 || sinks < 0)) return PKV_ERR_INVALID_ARG;
    if (scored) {
        // a cap far outside the scores' range would overflow score / softcap
        if (scored->softcap != 0.f && !(scored->softcap >= 1e-3f && scored->softcap <= 1e6f))
            return PKV_ERR_INVALID_ARG;
        if (window < 0 || ((reinterpret_cast<uintptr_t>(scored->slopes) | reinterpret_cast<uintptr_t>(scored->starts) |
                            reinterpret_cast<uintptr_t>(scored->prefix_lens)) & 3u))
            return PKV_ERR_INVALID_ARG;
    }
    if (num_seqs == 0 || num_rows == 0 || max_query_len == 0) return PKV_OK;
    if (!q || !out || !block_tables || !query_start || !context_lens || !pkv::aligned16(q) ||
        !pkv::aligned16(out))
        return PKV_ERR_INVALID_ARG;
    PrefillShape pp;
    // shape first (no CUDA call), then the plan for the real SM count
    pkv_status st = plan_prefill(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                 max_query_len, max_context_len, kv_splits, 1, &pp, window, has_prefix, sinks);
    if (st != PKV_OK) return st;
    int sm = 0;
    if (kv_splits == 0) {
        sm = pkv::current_sm_count();
        if (sm <= 0) return PKV_ERR_CUDA;
        st = plan_prefill(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_query_len,
                          max_context_len, 0, sm, &pp, window, has_prefix, sinks);
        if (st != PKV_OK) return st;
    }
    const bool plan_items = scored && planned(pp, num_seqs);
    const size_t partials = prefill_workspace(num_rows, num_q_heads, pp.splits);
    const size_t need = plan_items ? plan_bytes(pp, num_seqs) : partials;
    if (need > 0 && (!workspace || workspace_bytes < need || !pkv::aligned16(workspace)))
        return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    if (sm == 0) sm = pkv::current_sm_count();
    if (sm <= 0) return PKV_ERR_CUDA;
    const int group = num_q_heads / num_kv_heads;
    // the output has the queries' shape: full row tiles leave through the same boxes
    CUtensorMap tq, tk, tv, to;
    if (!pkv::encode_query_map(&tq, q, num_rows, num_q_heads, group, pp.tile_tokens, dtype) ||
        !pkv::encode_query_map(&to, out, num_rows, num_q_heads, group, pp.tile_tokens, dtype) ||
        !pkv::encode_half_map(&tk, k_cache, num_blocks, block_stride_elems, num_kv_heads, block_size,
                              dtype, 0) ||
        !pkv::encode_half_map(&tv, v_cache, num_blocks, block_stride_elems, num_kv_heads, block_size,
                              dtype, 0))
        return PKV_ERR_CUDA;

    pkv::PrefillParams p{};
    p.q = q;
    p.out = out;
    const size_t slots = static_cast<size_t>(num_rows) * num_q_heads * pp.splits;
    p.ws_o = partials ? static_cast<float *>(workspace) : nullptr;
    p.ws_m = partials ? p.ws_o + slots * head_dim : nullptr;
    p.ws_l = partials ? p.ws_m + slots : nullptr;
    p.block_tables = block_tables;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.status = status;
    p.num_blocks = num_blocks;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.len_cap = max_context_len;
    p.qlen_cap = max_query_len;
    p.num_rows = num_rows;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.tile_tokens = pp.tile_tokens;
    p.tile_rows = pp.tile_tokens * group;
    p.row_tiles = pp.row_tiles;
    p.num_items = pp.items;
    p.splits = pp.splits;
    p.split_tokens = pp.split_tokens;
    p.div_row_tiles = pkv::make_fast_div(p.row_tiles);
    p.div_kv_heads = pkv::make_fast_div(num_kv_heads);
    p.div_group = pkv::make_fast_div(group);
    p.div_splits = pkv::make_fast_div(p.splits);
    p.div_per_tile = pkv::make_fast_div(num_kv_heads * num_seqs * p.splits);
    // item order (prefill_item): whole prompts of one length (every chunk
    // max_query_len tokens on an empty cache) in row-tile pairs, a few sequences of
    // different lengths by (sequence, KV head) sorted by length, both for L2 reuse
    // of each (sequence, KV head)'s K/V tiles; otherwise row tiles, heaviest first
    const bool whole_prompts = num_rows == static_cast<int64_t>(num_seqs) * max_query_len &&
                               max_context_len == max_query_len;
    p.order = pp.splits != 1 ? pkv::kOrderRowTiles
              : whole_prompts ? pkv::kOrderPairs
              : num_seqs <= pkv::kSortedGroupsMaxSeqs ? pkv::kOrderSortedGroups
                                                      : pkv::kOrderRowTiles;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    if (scored) {
        p.slopes = scored->slopes;
        p.starts = scored->starts;
        p.prefix_lens = scored->prefix_lens;
        p.window = window;
        p.block_size = block_size;
        p.sinks = std::min(sinks, max_context_len);  // (rounded up to blocks in 32 bits)
        if (scored->softcap > 0.f) {
            p.cap_in = scale / scored->softcap;
            p.cap_out = static_cast<float>(scored->softcap * 1.4426950408889634);
            p.cap_short = p.cap_out <= 200.f;
            p.fixed_ref = dtype == PKV_BF16 && p.cap_out <= pkv::kFixedRefMax && !p.slopes;
            if (p.fixed_ref) p.shift = std::max(0.f, p.cap_out - pkv::kFixedWeightMax);
        }
    }
    // persistent: one CTA per SM (or per item when there are fewer)
    const int grid = std::min(pp.items, sm);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (plan_items) {
        auto *plan = static_cast<pkv::PrefillPlan *>(workspace);
        p.plan = plan;
        p.order = pkv::kOrderPlanned;
        if (pkv::launch_kernel(sink_form ? pkv::paged_prefill_plan_kernel<true> : pkv::paged_prefill_plan_kernel<false>, dim3(1),
                               dim3(pkv::kPlanThreads), 0, s, sink_form, p, plan) != cudaSuccess) {
            cudaGetLastError();
            return PKV_ERR_CUDA;
        }
        pkv::count_launch();
        if (st = pkv::launch_status(); st != PKV_OK) return st;
    }
    if (sink_form)
        return dtype == PKV_F16
                   ? pkv::launch_prefill_sinks_f16(p, tq, tk, tv, to, block_size, grid, max_query_len, s)
                   : pkv::launch_prefill_sinks_bf16(p, tq, tk, tv, to, block_size, grid, max_query_len, s);
    if (scored)
        return dtype == PKV_F16
                   ? pkv::launch_prefill_scored_f16(p, tq, tk, tv, to, block_size, grid, max_query_len, s)
                   : pkv::launch_prefill_scored_bf16(p, tq, tk, tv, to, block_size, grid, max_query_len, s);
    return dtype == PKV_F16
               ? pkv::launch_prefill<__half>(p, tq, tk, tv, to, block_size, grid, max_query_len, s)
               : pkv::launch_prefill<__nv_bfloat16>(p, tq, tk, tv, to, block_size, grid, max_query_len, s);
}

}  // namespace

extern "C" {

PKV_API size_t pkv_prefill_workspace_bytes(int num_rows, int num_seqs, int num_q_heads,
                                           int num_kv_heads, int head_dim, int block_size,
                                           int max_query_len, int max_context_len, int kv_splits) {
    const int sm = kv_splits > 0 ? 1 : pkv::current_sm_count();
    if (sm <= 0 || num_rows < 0) return static_cast<size_t>(-1);
    PrefillShape pp;
    if (plan_prefill(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_query_len,
                     max_context_len, kv_splits, sm, &pp) != PKV_OK)
        return static_cast<size_t>(-1);
    return prefill_workspace(num_rows, num_q_heads, pp.splits);
}

PKV_API pkv_status pkv_paged_attention_prefill(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, void *out, void *workspace, size_t workspace_bytes,
    int kv_splits, pkv_dtype dtype, void *stream) {
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_stride_elems, block_tables, max_blocks_per_seq,
                        query_start, context_lens, num_rows, max_query_len, max_context_len, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, scale, out, workspace,
                        workspace_bytes, kv_splits, dtype, stream, nullptr);
}

PKV_API size_t pkv_prefill_scored_workspace_bytes(int num_rows, int num_seqs, int num_q_heads,
                                                  int num_kv_heads, int head_dim, int block_size,
                                                  int max_query_len, int max_context_len, int window,
                                                  int has_prefix, int kv_splits) {
    const int sm = kv_splits > 0 ? 1 : pkv::current_sm_count();
    if (sm <= 0 || num_rows < 0 || window < 0) return static_cast<size_t>(-1);
    PrefillShape pp;
    if (plan_prefill(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_query_len,
                     max_context_len, kv_splits, sm, &pp, window, has_prefix != 0) != PKV_OK)
        return static_cast<size_t>(-1);
    if (planned(pp, num_seqs)) return plan_bytes(pp, num_seqs);
    return prefill_workspace(num_rows, num_q_heads, pp.splits);
}

PKV_API size_t pkv_prefill_sinks_workspace_bytes(int num_rows, int num_seqs, int num_q_heads, int num_kv_heads,
                                                 int head_dim, int block_size, int max_query_len, int max_context_len,
                                                 int window, int sinks, int kv_splits) {
    const int sm = kv_splits > 0 ? 1 : pkv::current_sm_count();
    if (sm <= 0 || num_rows < 0 || window < 1 || sinks < 0) return static_cast<size_t>(-1);
    PrefillShape pp;
    if (plan_prefill(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_query_len, max_context_len, kv_splits,
                     sm, &pp, window, false, sinks) != PKV_OK)
        return static_cast<size_t>(-1);
    if (planned(pp, num_seqs)) return plan_bytes(pp, num_seqs);
    return prefill_workspace(num_rows, num_q_heads, pp.splits);
}

PKV_API pkv_status pkv_paged_attention_prefill_sinks(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks, int64_t block_stride_elems,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_start, const int32_t *context_lens,
    int num_rows, int max_query_len, int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, int window, int sinks, void *out, void *workspace, size_t workspace_bytes, int kv_splits,
    pkv_dtype dtype, void *stream) {
    const ScoredPrefillArgs a{0.f, nullptr, window, nullptr, nullptr, true, sinks};
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_stride_elems, block_tables, max_blocks_per_seq,
                        query_start, context_lens, num_rows, max_query_len, max_context_len, num_seqs, num_q_heads,
                        num_kv_heads, head_dim, block_size, scale, out, workspace, workspace_bytes, kv_splits, dtype,
                        stream, &a);
}

PKV_API pkv_status pkv_paged_attention_prefill_scored(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, float softcap, const float *slopes, int window, const int32_t *starts,
    const int32_t *prefix_lens, void *out, void *workspace, size_t workspace_bytes, int kv_splits,
    pkv_dtype dtype, void *stream) {
    const ScoredPrefillArgs a{softcap, slopes, window, starts, prefix_lens};
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_stride_elems, block_tables, max_blocks_per_seq,
                        query_start, context_lens, num_rows, max_query_len, max_context_len, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, block_size, scale, out, workspace,
                        workspace_bytes, kv_splits, dtype, stream, &a);
}

}  // extern "C"
