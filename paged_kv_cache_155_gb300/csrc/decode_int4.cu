// decode_int4.cu -- the pkv_paged_attention_decode_int4 entry point: argument checks, the plan,
// workspace layout, and the launch.
#include <algorithm>
#include <cmath>

#include "decode_int4_launch.cuh"

namespace {

constexpr int kWorkersPerCta = 4;

struct Int4Plan {
    int heads = 8;     // heads per block: 4, 8 or 16
    int blocks = 1;    // blocks of heads per KV head
    int resident = 3;  // CTAs per SM (DecodeInt4Geom::kResident)
};

pkv_status plan_int4(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
                     Int4Plan *plan) {
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || max_context_len < 0)
        return PKV_ERR_INVALID_ARG;
    // the fewest blocks of at most 16 heads that cover the group, of 4 or 8 heads where these do
    const int group = num_q_heads / num_kv_heads;
    plan->blocks = (group + 15) / 16;
    const int each = (group + plan->blocks - 1) / plan->blocks;
    plan->heads = each <= 4 ? 4 : each <= 8 ? 8 : 16;
    plan->blocks = (group + plan->heads - 1) / plan->heads;
    plan->resident = plan->heads <= 8 ? (head_dim == 64 ? 4 : 3) : (head_dim == 64 ? 3 : 2);
    // all units' chunks fit the kernel's 32-bit count
    const int64_t units = static_cast<int64_t>(num_kv_heads) * plan->blocks;
    const int64_t chunks = std::max<int64_t>(1, (max_context_len + 31LL) / 32);
    if (units > 0x3fffffff || units * chunks > 0x3fffffff || units * chunks * std::max(num_seqs, 1) > 0x3fffffff)
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

// Workspace: the partials of two pieces per worker, then what the merge has to know per worker.
size_t workspace_of(const Int4Plan &plan, int head_dim, int sm_count) {
    const size_t workers = static_cast<size_t>(sm_count) * plan.resident * kWorkersPerCta;
    return workers * (2 * plan.heads * (static_cast<size_t>(head_dim) + 2) * sizeof(float) + sizeof(pkv::Int4Split));
}

}  // namespace

extern "C" {

PKV_API size_t pkv_decode_int4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                               int block_size, int max_context_len) {
    Int4Plan plan;
    if (plan_int4(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &plan) != PKV_OK)
        return static_cast<size_t>(-1);
    const int sm = pkv::current_sm_count();
    return sm > 0 ? workspace_of(plan, head_dim, sm) : static_cast<size_t>(-1);
}

PKV_API pkv_status pkv_paged_attention_decode_int4(const void *q, const void *k_cache, const void *v_cache,
                                                   int64_t num_blocks, int64_t block_stride_bytes,
                                                   const int32_t *block_tables, int max_blocks_per_seq,
                                                   const int32_t *context_lens, int max_context_len, int num_seqs,
                                                   int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                   float scale, void *out, void *workspace, size_t workspace_bytes,
                                                   pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    Int4Plan plan;
    const pkv_status st = plan_int4(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &plan);
    if (st != PKV_OK) return st;
    if (num_blocks <= 0 || num_blocks > 0x7fffffffLL || max_blocks_per_seq <= 0 ||
        static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    const int64_t half = static_cast<int64_t>(num_kv_heads) * pkv::int4_record_bytes(head_dim, block_size);
    if (block_stride_bytes < half || block_stride_bytes % 16) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !out || !block_tables || !context_lens || !workspace || !pkv::aligned16(q) || !pkv::aligned16(out) ||
        !pkv::aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens)) & 3u))
        return PKV_ERR_INVALID_ARG;
    const int sm = pkv::current_sm_count();
    if (sm <= 0) return PKV_ERR_CUDA;
    if (workspace_bytes < workspace_of(plan, head_dim, sm)) return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;

    pkv::Int4Params p{};
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.out = out;
    const size_t rows = static_cast<size_t>(sm) * plan.resident * kWorkersPerCta * 2 * plan.heads;
    p.seg_o = static_cast<float *>(workspace);
    p.seg_m = p.seg_o + rows * head_dim;
    p.seg_l = p.seg_m + rows;
    p.splits = reinterpret_cast<pkv::Int4Split *>(p.seg_l + rows);
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
    p.blocks = plan.blocks;
    p.units = num_kv_heads * plan.blocks;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    // every SM's resident CTAs, or fewer where the contexts' bound leaves no more shares
    const int64_t chunks = std::max<int64_t>(1, (max_context_len + 31LL) / 32) * p.units * num_seqs;
    const int64_t most = (chunks + pkv::kInt4MinShare * kWorkersPerCta - 1) / (pkv::kInt4MinShare * kWorkersPerCta);
    const int grid = static_cast<int>(std::min<int64_t>(most, static_cast<int64_t>(sm) * plan.resident));
    p.seg_workers = sm * plan.resident * kWorkersPerCta;
    p.by_unit = static_cast<int64_t>(num_seqs) * p.units <= static_cast<int64_t>(grid) * kWorkersPerCta;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == PKV_F16 ? pkv::launch_int4_f16(p, head_dim, block_size, plan.heads, grid, s)
                            : pkv::launch_int4_bf16(p, head_dim, block_size, plan.heads, grid, s);
}

}  // extern "C"
