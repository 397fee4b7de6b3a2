// tree.cu -- a tree of drafted tokens over the paged cache:
//   pkv_paged_attention_tree  the verification's attention: argument checks, workspace and launches
//                             (kernel: paged_prefill_tc_kernel, tree form)
//   pkv_tree_commit           the accepted path's K/V rows moved together
#include <algorithm>
#include <cmath>

#include "prefill_launch.cuh"

namespace {

// Workspace: the partials of two pieces per CTA, then what the merge has to know per CTA.
constexpr size_t kSegRows = 2 * 128;
size_t tree_workspace(int sm_count) {
    return static_cast<size_t>(sm_count) * (kSegRows * (128 + 2) * sizeof(float) + sizeof(pkv::TreeSplit));
}

struct CommitParams {
    char *k_cache, *v_cache;
    const int32_t *block_tables, *query_start, *context_lens, *accepted, *accepted_lens;
    int32_t *new_context_lens;
    unsigned int *status;
    int64_t num_blocks, block_stride;  // bytes
    int max_blocks_per_seq, len_cap, qlen_cap, num_kv_heads, row_vecs, block_shift, max_accepted;
};

constexpr int kCommitThreads = 128;
constexpr int kCommitDepth = 8;

// (Launched ahead, it waits for the attention before it: write, attention and commit of 8 x 16 nodes 35.5 us, not 39.8.)
// One thread per 16-byte column of a head's rows (K and V, grid.y): it walks the path's nodes in
// order, so that a row is read before a later node's move could overwrite it -- node j goes to
// place j, and nodes ascend, so place j is never the source of a node behind j -- and only its own
// column, so no other thread is in the way.  kCommitDepth rows are in flight together: those are
// loaded before any of them is stored.
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitParams p) {
    pkv::pdl_trigger();
    pkv::pdl_wait();
    const int seq = blockIdx.z;
    const int q0 = p.query_start[seq], q1 = p.query_start[seq + 1], len = p.context_lens[seq];
    const bool lead = threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0;
    // (compared before they are subtracted: any values may stand here)
    if (q0 < 0 || q1 < q0 || q1 - q0 > p.qlen_cap || len < q1 - q0 || len > p.len_cap) {
        if (lead) pkv::raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        if (lead && p.new_context_lens) p.new_context_lens[seq] = len;
        return;
    }
    const int chunk = q1 - q0, base = len - chunk;
    int n = p.accepted_lens[seq];
    if (n < 0 || n > p.max_accepted || n > chunk) {
        if (lead) pkv::raise_flag(p.status, PKV_DEVERR_KEPT);
        n = 0;
    }
    const int32_t *path = p.accepted + static_cast<int64_t>(seq) * p.max_accepted;
    const int32_t *table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
    const int bs = 1 << p.block_shift;
    const int c = blockIdx.x * kCommitThreads + threadIdx.x;
    const bool mine = c < p.num_kv_heads * p.row_vecs;
    const int head = c / p.row_vecs, vec = c - head * p.row_vecs;
    char *cache = (blockIdx.y ? p.v_cache : p.k_cache) + vec * 16;
    // -1: a flagged table entry
    auto row_of = [&](int t) -> int64_t {
        const int b = table[t >> p.block_shift];
        if (b < 0 || b >= p.num_blocks) {
            if (lead) pkv::raise_flag(p.status, PKV_DEVERR_BLOCK_TABLE);
            return -1;
        }
        return b * p.block_stride + (static_cast<int64_t>(head) * bs + (t & (bs - 1))) * p.row_vecs * 16;
    };
    int before = -1;  // the path's last node
    for (int j0 = 0; j0 < n; j0 += kCommitDepth) {
        uint4 row[kCommitDepth];
        int64_t to[kCommitDepth];
#pragma unroll
        for (int k = 0; k < kCommitDepth; ++k) {
            to[k] = -1;
            const int j = j0 + k;
            if (j >= n) continue;
            const int node = path[j];
            if (node <= before || node >= chunk) {  // (ascending from 0 on: node >= j)
                if (lead) pkv::raise_flag(p.status, PKV_DEVERR_KEPT);
                continue;
            }
            before = node;
            if (node == j) continue;  // in its place
            const int64_t src = row_of(base + node), dst = row_of(base + j);
            if (src < 0 || dst < 0 || !mine) continue;
            row[k] = *reinterpret_cast<const uint4 *>(cache + src);
            to[k] = dst;
        }
#pragma unroll
        for (int k = 0; k < kCommitDepth; ++k)
            if (to[k] >= 0) *reinterpret_cast<uint4 *>(cache + to[k]) = row[k];
    }
    if (lead && p.new_context_lens) p.new_context_lens[seq] = base + n;
}

}  // namespace

extern "C" {

PKV_API size_t pkv_tree_workspace_bytes(void) {
    const int sm = pkv::current_sm_count();
    return sm > 0 ? tree_workspace(sm) : static_cast<size_t>(-1);
}

PKV_API pkv_status pkv_paged_attention_tree(const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
                                            int64_t block_stride_elems, const int32_t *block_tables,
                                            int max_blocks_per_seq, const int32_t *query_start,
                                            const int32_t *context_lens, const int64_t *tree_mask, int mask_words,
                                            int num_rows, int max_query_len, int max_context_len, int num_seqs,
                                            int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                                            void *out, void *workspace, size_t workspace_bytes, pkv_dtype dtype,
                                            void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        num_kv_heads > 65535 || num_blocks <= 0 || num_blocks > 0x7fffffffLL || max_blocks_per_seq <= 0 ||
        max_query_len < 0 || max_context_len < max_query_len ||
        static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size ||
        mask_words < 0 || mask_words > (1 << 20) || static_cast<int64_t>(mask_words) * 64 < max_query_len || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads;
    if (group > 128) return PKV_ERR_UNSUPPORTED;  // a row tile holds at least one token
    const int64_t half_elems = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_elems < half_elems || block_stride_elems % 8) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_rows == 0 || max_query_len == 0) return PKV_OK;
    // all units' KV tiles fit the kernel's 32-bit count
    const int tile_tokens = 128 / group;
    const int64_t tiles = (max_context_len + 127LL) / 128, row_tiles = (max_query_len + tile_tokens - 1LL) / tile_tokens;
    if (tiles * row_tiles > 0x3fffffff || tiles * row_tiles * num_kv_heads > 0x3fffffff ||
        tiles * row_tiles * num_kv_heads * num_seqs > 0x3fffffff)
        return PKV_ERR_INVALID_ARG;
    if (!q || !out || !block_tables || !query_start || !context_lens || !tree_mask || !workspace || !pkv::aligned16(q) ||
        !pkv::aligned16(out) || !pkv::aligned16(workspace) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(query_start) |
          reinterpret_cast<uintptr_t>(context_lens)) & 3u))
        return PKV_ERR_INVALID_ARG;
    const int sm = pkv::current_sm_count();
    if (sm <= 0) return PKV_ERR_CUDA;
    if (workspace_bytes < tree_workspace(sm)) return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    CUtensorMap tq, tk, tv, to;
    if (!pkv::encode_query_map(&tq, q, num_rows, num_q_heads, group, tile_tokens, dtype) ||
        !pkv::encode_query_map(&to, out, num_rows, num_q_heads, group, tile_tokens, dtype) ||
        !pkv::encode_half_map(&tk, k_cache, num_blocks, block_stride_elems, num_kv_heads, block_size, dtype, 0) ||
        !pkv::encode_half_map(&tv, v_cache, num_blocks, block_stride_elems, num_kv_heads, block_size, dtype, 0))
        return PKV_ERR_CUDA;
    pkv::PrefillParams p{};
    p.q = q;
    p.out = out;
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
    p.tile_tokens = tile_tokens;
    p.tile_rows = tile_tokens * group;
    p.splits = 1;
    p.order = pkv::kOrderStream;
    p.block_size = block_size;
    p.div_kv_heads = pkv::make_fast_div(num_kv_heads);
    p.div_group = pkv::make_fast_div(group);
    p.div_tile_tokens = pkv::make_fast_div(tile_tokens);
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    p.tree_mask = tree_mask;
    p.mask_words = mask_words;
    p.seg_o = static_cast<float *>(workspace);
    p.seg_m = p.seg_o + static_cast<size_t>(sm) * kSegRows * 128;
    p.seg_l = p.seg_m + static_cast<size_t>(sm) * kSegRows;
    p.tree_splits = reinterpret_cast<pkv::TreeSplit *>(p.seg_l + static_cast<size_t>(sm) * kSegRows);
    // one CTA per SM, or fewer where the contexts' bound leaves no more shares
    p.abreast = row_tiles > 1 && num_kv_heads % 2 == 0 && sm > 1 ? 2 : 1;
    const int64_t most = (tiles * row_tiles * num_kv_heads * num_seqs / p.abreast + pkv::kMinShare - 1) / pkv::kMinShare;
    const int grid = static_cast<int>(std::min<int64_t>(most, sm / p.abreast)) * p.abreast;
    p.row_tiles = static_cast<int>(row_tiles);
    p.by_unit = row_tiles * num_kv_heads * num_seqs <= grid;
    p.seg_ctas = sm;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == PKV_F16 ? pkv::launch_tree_f16(p, tq, tk, tv, to, block_size, grid, s)
                            : pkv::launch_tree_bf16(p, tq, tk, tv, to, block_size, grid, s);
}

PKV_API pkv_status pkv_tree_commit(void *k_cache, void *v_cache, int64_t num_blocks, int64_t block_stride_elems,
                                   int num_kv_heads, int head_dim, int block_size, const int32_t *block_tables,
                                   int max_blocks_per_seq, const int32_t *query_start, const int32_t *context_lens,
                                   int max_query_len, int max_context_len, int num_seqs, const int32_t *accepted,
                                   const int32_t *accepted_lens, int max_accepted, int32_t *new_context_lens,
                                   pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16 && dtype != PKV_INT8) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    const int elem = dtype == PKV_INT8 ? 1 : 2;
    if (num_seqs < 0 || num_seqs > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks <= 0 ||
        num_blocks > 0x7fffffffLL || max_blocks_per_seq <= 0 || max_query_len < 0 || max_context_len < max_query_len ||
        static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size || max_accepted < 0)
        return PKV_ERR_INVALID_ARG;
    const int64_t half_elems = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_elems < half_elems || block_stride_elems * elem % 16) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !query_start || !context_lens || !accepted_lens || (!accepted && max_accepted > 0) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(query_start) |
          reinterpret_cast<uintptr_t>(context_lens) | reinterpret_cast<uintptr_t>(accepted) |
          reinterpret_cast<uintptr_t>(accepted_lens) | reinterpret_cast<uintptr_t>(new_context_lens)) & 3u))
        return PKV_ERR_INVALID_ARG;
    // every CTA of a sequence reads its entries of these: the new lengths need a place of their own
    auto meets = [&](const int32_t *in, int64_t count) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(new_context_lens);
        return a < b + 4 * static_cast<uintptr_t>(num_seqs) && b < a + 4 * static_cast<uintptr_t>(count);
    };
    const int64_t seqs = num_seqs;
    if (new_context_lens && (meets(context_lens, seqs) || meets(query_start, seqs + 1) || meets(accepted_lens, seqs) ||
                             meets(accepted, seqs * max_accepted) || meets(block_tables, seqs * max_blocks_per_seq)))
        return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    const int row_vecs = head_dim * elem / 16;
    CommitParams p{static_cast<char *>(k_cache), static_cast<char *>(v_cache), block_tables, query_start, context_lens,
                   accepted, accepted_lens, new_context_lens, status, num_blocks, block_stride_elems * elem,
                   max_blocks_per_seq, max_context_len, max_query_len, num_kv_heads, row_vecs,
                   block_size == 8 ? 3 : block_size == 16 ? 4 : 5, max_accepted};
    const int cols = num_kv_heads * row_vecs;
    const dim3 grid(static_cast<unsigned>((cols + kCommitThreads - 1) / kCommitThreads), 2, static_cast<unsigned>(num_seqs));
    if (pkv::launch_kernel(tree_commit_kernel, grid, dim3(kCommitThreads), 0, static_cast<cudaStream_t>(stream), true, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    pkv::count_launch();
    return pkv::launch_status();
}

}  // extern "C"
