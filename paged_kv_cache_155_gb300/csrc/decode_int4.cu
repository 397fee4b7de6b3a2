// decode_int4.cu -- the pkv_paged_attention_decode_int4 entry point: argument checks, the
// split-context plan, workspace layout, and the launch.
#include <algorithm>
#include <cmath>

#include "decode_int4_launch.cuh"

namespace {

constexpr int kMinPartition = 256;  // tokens
// What starting and ending a CTA costs, in tokens of its main loop.
constexpr int kCtaTokens = 128;
constexpr int kMaxWaves = 8;        // waves of resident CTAs that a split may make

struct Int4Plan {
    int partition = 0, partitions = 1, tiles = 1, blocks = 1;  // tiles of 8 heads per block, blocks per KV head
};

pkv_status plan_int4(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
                     int partition_size, int sm_count, Int4Plan *plan) {
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || max_context_len < 0 ||
        partition_size < 0 || sm_count <= 0 || partition_size % 32)
        return PKV_ERR_INVALID_ARG;
    constexpr int kEntries = pkv::DecodeInt4Geom<128, 16, 1>::kMaxTableEntries;
    const int most = kEntries * block_size;
    if (partition_size > most) return PKV_ERR_INVALID_ARG;
    // the fewest blocks of at most 16 heads that cover the group, of 8 heads where these do
    const int group = num_q_heads / num_kv_heads;
    plan->blocks = (group + 15) / 16;
    plan->tiles = (group + plan->blocks - 1) / plan->blocks <= 8 ? 1 : 2;
    plan->blocks = (group + 8 * plan->tiles - 1) / (8 * plan->tiles);
    const int64_t grid_y = static_cast<int64_t>(num_kv_heads) * plan->blocks;
    if (grid_y > 65535 || num_seqs > 65535) return PKV_ERR_INVALID_ARG;
    const int64_t len = std::max(1, max_context_len);
    auto part_for = [&](int64_t n) { return ((len + n - 1) / n + 31) / 32 * 32; };
    int64_t part = partition_size;
    if (part == 0) {
        // The split whose rounds of resident CTAs take the least time for sequences of the
        // longest length: rounds x (a partition's tokens + a CTA's fixed cost).
        const int64_t units = std::max<int64_t>(1, num_seqs * grid_y);
        const int64_t slots = static_cast<int64_t>(sm_count) * (plan->tiles == 1 ? 3 : 2);
        const int64_t fewest = (len + most - 1) / most;
        const int64_t most_parts = std::max(fewest, std::min((len + kMinPartition - 1) / kMinPartition,
                                                             (kMaxWaves * slots + units - 1) / units));
        // (for w rounds, the most partitions that still take w)
        int64_t best = -1;
        for (int w = 0; w <= kMaxWaves + 1; ++w) {
            const int64_t n = w == 0 ? fewest : w > kMaxWaves ? most_parts : std::max(fewest, std::min(most_parts, w * slots / units));
            const int64_t p = part_for(n), parts = (len + p - 1) / p;
            if (p > most) continue;
            const int64_t cost = (units * parts + slots - 1) / slots * (p + kCtaTokens);
            if (best < 0 || cost < best) {
                best = cost;
                part = p;
            }
        }
        if (part == 0) part = most;
    }
    plan->partition = static_cast<int>(part);
    plan->partitions = static_cast<int>((len + part - 1) / part);
    return PKV_OK;
}

size_t workspace_of(int num_seqs, int num_q_heads, int head_dim, int partitions) {
    if (partitions <= 1) return 0;
    return static_cast<size_t>(num_seqs) * num_q_heads * partitions * (static_cast<size_t>(head_dim) + 2) * sizeof(float);
}

}  // namespace

extern "C" {

PKV_API size_t pkv_decode_int4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                               int block_size, int max_context_len, int partition_size) {
    const int sm = partition_size > 0 ? 1 : pkv::current_sm_count();
    if (sm <= 0) return static_cast<size_t>(-1);
    Int4Plan plan;
    if (plan_int4(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size, sm, &plan) != PKV_OK)
        return static_cast<size_t>(-1);
    return workspace_of(num_seqs, num_q_heads, head_dim, plan.partitions);
}

PKV_API pkv_status pkv_paged_attention_decode_int4(const void *q, const void *k_cache, const void *v_cache,
                                                   int64_t num_blocks, int64_t block_stride_bytes,
                                                   const int32_t *block_tables, int max_blocks_per_seq,
                                                   const int32_t *context_lens, int max_context_len, int num_seqs,
                                                   int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                   float scale, void *out, void *workspace, size_t workspace_bytes,
                                                   int partition_size, pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    Int4Plan plan;
    // shape first (no CUDA call), then the plan for the real SM count
    pkv_status st = plan_int4(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size, 1, &plan);
    if (st != PKV_OK) return st;
    if (num_blocks <= 0 || num_blocks > 0x7fffffffLL || max_blocks_per_seq <= 0 ||
        static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    const int64_t half = static_cast<int64_t>(num_kv_heads) * pkv::int4_record_bytes(head_dim, block_size);
    if (block_stride_bytes < half || block_stride_bytes % 16) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !out || !block_tables || !context_lens || !pkv::aligned16(q) || !pkv::aligned16(out) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens)) & 3u))
        return PKV_ERR_INVALID_ARG;
    if (partition_size == 0) {
        const int sm = pkv::current_sm_count();
        if (sm <= 0) return PKV_ERR_CUDA;
        st = plan_int4(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, 0, sm, &plan);
        if (st != PKV_OK) return st;
    }
    const size_t need = workspace_of(num_seqs, num_q_heads, head_dim, plan.partitions);
    if (need > 0 && (!workspace || workspace_bytes < need || !pkv::aligned16(workspace))) return PKV_ERR_INVALID_ARG;
    if (plan.partitions > 1 && static_cast<int64_t>(num_seqs) * num_q_heads > 0x7fffffff) return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;

    pkv::DecodeParams p{};
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.out = out;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * plan.partitions;
    p.ws_o = need ? static_cast<float *>(workspace) : nullptr;
    p.ws_m = need ? p.ws_o + rows * head_dim : nullptr;
    p.ws_l = need ? p.ws_m + rows : nullptr;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = status;
    p.num_blocks = num_blocks;
    p.block_stride = block_stride_bytes;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.len_cap = max_context_len;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.group = num_q_heads / num_kv_heads;
    p.subgroups = plan.blocks;
    p.items_y = num_kv_heads * plan.blocks;
    p.partition_size = plan.partition;
    p.num_partitions = plan.partitions;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    const int merge_rows = plan.partitions > 1 ? num_seqs * num_q_heads : 0;
    p.trigger_dependents = merge_rows > 0;
    const dim3 grid(static_cast<unsigned>(plan.partitions), static_cast<unsigned>(p.items_y), static_cast<unsigned>(num_seqs));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == PKV_F16 ? pkv::launch_int4_f16(p, head_dim, block_size, plan.tiles, grid, merge_rows, s)
                            : pkv::launch_int4_bf16(p, head_dim, block_size, plan.tiles, grid, merge_rows, s);
}

}  // extern "C"
