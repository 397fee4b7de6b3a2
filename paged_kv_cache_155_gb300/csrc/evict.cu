// evict.cu -- eviction from the paged cache by accumulated attention weight:
//   pkv_evict_select   which tokens of each (sequence, KV head) stay
//   pkv_evict_compact  their K/V rows to the front of the sequence's context
//
// The weights are what pkv_paged_attention_decode_scored accumulates: per KV head
// and cached token, the softmax weight that the group's queries gave the token.
// Each KV head keeps its own tokens; every head keeps the same number, so one block
// table and one context length still describe the sequence.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace {

// ------------------------------------------------------------------ select
// Order-preserving map of a weight to an unsigned key: larger weight, larger key;
// -0 equals +0; NaN sorts lowest.  Key 0 is NaN's alone.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectParams {
    const float *weights;  // [num_seqs][num_kv_heads][weights_stride]
    float *weights_out;    // null, or the same shape (may be `weights` itself)
    const int32_t *context_lens;
    int32_t *kept;         // [num_seqs][num_kv_heads][budget]
    int32_t *kept_lens;    // [num_seqs]
    unsigned int *status;
    int64_t weights_stride;
    int len_cap, budget, sinks, recent, num_kv_heads;
};

// One CTA per (KV head, sequence).  The kept tokens are the first `sinks`, the last
// `recent` and, of those between, the `need` heaviest, equal weights by lower index.
// The threshold -- the need-th largest key -- is found two bits at a time from the
// top: count the keys at or above three candidate prefixes and descend.  Counting
// needs no order and no shared-memory atomics (weights crowd into few exponents, so
// histogram bins would collide), and stops as soon as a prefix holds exactly `need`
// keys.  Keys of the first R x THREADS tokens stay in registers; a longer row's
// others are read again (from L2) in each step.  The kept positions then leave in
// ascending order, EB x THREADS tokens at a time, by a block-wide prefix count.
template <int THREADS, int R>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const SelectParams p) {
    constexpr int WARPS = THREADS / 32, HELD = R * THREADS, EB = R < 8 ? R : 8, BATCH = EB * THREADS;
    __shared__ uint32_t counts[2][3][WARPS];
    __shared__ uint32_t totals[EB * WARPS];  // (kept outright, ties) of each 32 tokens, 16 bits each
    __shared__ uint32_t bases[EB * WARPS];   // their exclusive prefix
    __shared__ uint32_t batch_total;
    const int h = blockIdx.x, seq = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = static_cast<int64_t>(seq) * p.num_kv_heads + h;
    int len = p.context_lens[seq];
    if (len < 0 || len > p.len_cap) {
        if (tid == 0 && h == 0) pkv::raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        len = len < 0 ? 0 : p.len_cap;
    }
    const int keep = min(len, p.budget);
    if (h == 0 && tid == 0) p.kept_lens[seq] = keep;
    const float *w = p.weights + row * p.weights_stride;
    float *wout = p.weights_out ? p.weights_out + row * p.weights_stride : nullptr;
    int32_t *kept = p.kept + row * p.budget;
    for (int i = keep + tid; i < p.budget; i += THREADS) kept[i] = -1;
    const bool all = len <= p.budget;
    const int mid0 = p.sinks, mid1 = len - p.recent;  // the tokens that compete, when !all
    const uint32_t need = all ? 0u : static_cast<uint32_t>(p.budget - p.sinks - p.recent);

    // the largest prefix `thr` with at least `need` keys at or above it
    uint32_t thr = 0u, ties = 0u;
    bool exact = false;  // exactly `need` keys are at or above thr
    if (need > 0) {
        uint32_t key[R];  // of token r * THREADS + tid; 0 outside the competing tokens
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r * THREADS + tid;
            key[r] = (t >= mid0 && t < mid1) ? __float_as_uint(w[t]) : 0xffffffffu;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = weight_key(__uint_as_float(key[r]));  // (all ones is a NaN: key 0)
        auto count_above = [&](auto above) {  // sum of above(key) over this thread's keys
#pragma unroll
            for (int r = 0; r < R; ++r) above(key[r]);
            for (int t = HELD + tid; t < mid1; t += THREADS)
                if (t >= mid0) above(weight_key(w[t]));
        };
        int buf = 0;
        for (int shift = 30; shift >= 0 && !exact; shift -= 2, buf ^= 1) {
            uint32_t n[3] = {0u, 0u, 0u};
            const uint32_t c1 = thr + (1u << shift), c2 = thr + (2u << shift), c3 = thr + (3u << shift);
            count_above([&](uint32_t k) {
                n[0] += k >= c1;
                n[1] += k >= c2;
                n[2] += k >= c3;
            });
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                n[i] = __reduce_add_sync(0xffffffffu, n[i]);
                if (lane == 0) counts[buf][i][warp] = n[i];
            }
            __syncthreads();  // the other buffer is rewritten only after the next one
#pragma unroll
            for (int i = 0; i < 3; ++i) n[i] = __reduce_add_sync(0xffffffffu, lane < WARPS ? counts[buf][i][lane] : 0u);
            const int step = n[2] >= need ? 3 : n[1] >= need ? 2 : n[0] >= need ? 1 : 0;
            thr += static_cast<uint32_t>(step) << shift;
            exact = step > 0 && n[step > 0 ? step - 1 : 0] == need;
        }
        if (!exact) {
            // thr is the need-th largest key itself: the keys above it stay, and of those
            // equal to it the first `ties`
            uint32_t n = 0u;
            count_above([&](uint32_t k) { n += k > thr; });
            n = __reduce_add_sync(0xffffffffu, n);
            __syncthreads();
            if (lane == 0) counts[0][0][warp] = n;
            __syncthreads();
            ties = need - __reduce_add_sync(0xffffffffu, lane < WARPS ? counts[0][0][lane] : 0u);
        }
    }

    uint32_t done = 0u, ties_done = 0u;  // tokens kept outright / equal to the threshold, before this batch
    for (int t0 = 0; t0 < len; t0 += BATCH) {
        float val[EB];
#pragma unroll
        for (int r = 0; r < EB; ++r) {
            const int t = t0 + r * THREADS + tid;
            val[r] = t < len ? w[t] : 0.f;
        }
        uint32_t in_mask[EB], tie_mask[EB];  // the warp's tokens r: stays outright / equals the threshold
#pragma unroll
        for (int r = 0; r < EB; ++r) {
            const int t = t0 + r * THREADS + tid;
            const uint32_t k = weight_key(val[r]);
            const bool fixed = t < len && (all || t < mid0 || t >= mid1);
            const bool competes = need > 0 && t >= mid0 && t < mid1;
            in_mask[r] = __ballot_sync(0xffffffffu, fixed || (competes && (exact ? k >= thr : k > thr)));
            tie_mask[r] = __ballot_sync(0xffffffffu, competes && !exact && k == thr);
            if (lane == 0) totals[r * WARPS + warp] = __popc(in_mask[r]) | (__popc(tie_mask[r]) << 16);
        }
        __syncthreads();
        if (warp == 0) {  // each half of a sum stays below 2^16
            constexpr int PER = (EB * WARPS + 31) / 32;
            uint32_t local[PER], sum = 0u;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = lane * PER + i;
                local[i] = sum;
                sum += at < EB * WARPS ? totals[at] : 0u;
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = lane * PER + i;
                if (at < EB * WARPS) bases[at] = incl - sum + local[i];
            }
            if (lane == 31) batch_total = incl;
        }
        __syncthreads();
        // ranks only move tokens down, and every weight of this batch is in registers:
        // weights_out may be weights
#pragma unroll
        for (int r = 0; r < EB; ++r) {
            const uint32_t before = bases[r * WARPS + warp], mask = (1u << lane) - 1u;
            const uint32_t in_before = done + (before & 0xffffu) + __popc(in_mask[r] & mask);
            const uint32_t tie_before = ties_done + (before >> 16) + __popc(tie_mask[r] & mask);
            if (((in_mask[r] >> lane) & 1u) || (((tie_mask[r] >> lane) & 1u) && tie_before < ties)) {
                const uint32_t rank = in_before + min(tie_before, ties);
                kept[rank] = t0 + r * THREADS + tid;
                if (wout) wout[rank] = val[r];
            }
        }
        done += batch_total & 0xffffu;
        ties_done += batch_total >> 16;
        __syncthreads();  // before the next batch rewrites the shared counts
    }
    if (wout)
        for (int i = keep + tid; i < len; i += THREADS) wout[i] = 0.f;  // slots the next tokens take
}

// ------------------------------------------------------------------ compact
struct CompactParams {
    char *k_cache, *v_cache;
    const int32_t *src_tables;  // [num_seqs][src_stride]
    const int32_t *dst_tables;  // [num_seqs][dst_stride]
    const int32_t *context_lens, *kept, *kept_lens;
    unsigned int *status;
    int64_t num_blocks, block_stride;  // bytes
    int src_stride, dst_stride, budget, num_kv_heads, block_size, src_cap, dst_cap;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// The bytes of token row (block, head, offset) of one pool half.
__device__ __forceinline__ int64_t row_offset(const CompactParams &p, int blk, int h, int t, int row_bytes) {
    return static_cast<int64_t>(blk) * p.block_stride + (static_cast<int64_t>(h) * p.block_size + t % p.block_size) * row_bytes;
}

// Moves token row kept[i] to position i.  VECS 16-byte vectors of a row per CTA
// column group; grid: (tiles x column groups x 2 halves, KV head, sequence).
// Into fresh blocks (IN_PLACE false) the tiles are independent.  In place, a CTA
// walks its column group's tiles in ascending order: kept[i] >= i and kept ascends,
// so a tile's stores (positions [a, b)) can only meet rows that tiles up to this one
// read, never a later tile's sources -- one barrier between a tile's loads and its
// stores orders them, and column groups never meet.
template <int ROW_VECS, int VECS, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
    constexpr int ROWS = kMoveThreads / VECS, TILE = ROWS * kMoveUnroll, GROUPS = ROW_VECS / VECS;
    const int h = blockIdx.y, seq = blockIdx.z;
    const int half = blockIdx.x % 2, group = (blockIdx.x / 2) % GROUPS, tile0 = blockIdx.x / (2 * GROUPS);
    int len = p.context_lens[seq], n = p.kept_lens[seq];
    const bool first = threadIdx.x == 0 && blockIdx.x == 0 && h == 0;
    if (len < 0 || len > p.src_cap || n < 0 || n > p.budget || n > len || n > p.dst_cap) {
        if (first) pkv::raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        return;  // uniform over the sequence's CTAs
    }
    char *base = half ? p.v_cache : p.k_cache;
    const int col = (group * VECS + threadIdx.x % VECS) * 16, row0 = threadIdx.x / VECS;
    const int32_t *kept = p.kept + (static_cast<int64_t>(seq) * p.num_kv_heads + h) * p.budget;
    const int32_t *src_table = p.src_tables + static_cast<int64_t>(seq) * p.src_stride;
    const int32_t *dst_table = p.dst_tables + static_cast<int64_t>(seq) * p.dst_stride;
    const int step = IN_PLACE ? TILE : n;  // out of place: this tile alone
    for (int i0 = tile0 * TILE; i0 < n; i0 += step) {
        uint4 x[kMoveUnroll];
        int64_t to[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = i0 + u * ROWS + row0;
            to[u] = -1;
            if (i >= n) continue;
            const int t = kept[i];
            if (IN_PLACE && t == i) continue;  // already there
            if (t < 0 || t >= len || (IN_PLACE && t < i)) {
                pkv::raise_flag(p.status, PKV_DEVERR_KEPT);
                continue;
            }
            const int sb = src_table[t / p.block_size], db = dst_table[i / p.block_size];
            if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
                pkv::raise_flag(p.status, PKV_DEVERR_BLOCK_TABLE);
                continue;
            }
            x[u] = *reinterpret_cast<const uint4 *>(base + row_offset(p, sb, h, t, ROW_VECS * 16) + col);
            to[u] = row_offset(p, db, h, i, ROW_VECS * 16) + col;
        }
        if (IN_PLACE) __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (to[u] >= 0) *reinterpret_cast<uint4 *>(base + to[u]) = x[u];
        if (!IN_PLACE) break;
    }
}

template <int ROW_VECS>
void launch_compact(const CompactParams &p, bool in_place, int max_kept, int num_seqs, cudaStream_t s) {
    if (in_place) {
        constexpr int VECS = ROW_VECS < 4 ? ROW_VECS : 4;  // 64-byte columns: more chains, whole sectors
        const dim3 grid(2 * (ROW_VECS / VECS), p.num_kv_heads, num_seqs);
        evict_compact_kernel<ROW_VECS, VECS, true><<<grid, kMoveThreads, 0, s>>>(p);
    } else {
        constexpr int TILE = kMoveThreads / ROW_VECS * kMoveUnroll;
        const dim3 grid(2 * ((max_kept + TILE - 1) / TILE), p.num_kv_heads, num_seqs);
        evict_compact_kernel<ROW_VECS, ROW_VECS, false><<<grid, kMoveThreads, 0, s>>>(p);
    }
}

}  // namespace

extern "C" {

PKV_API pkv_status pkv_evict_select(const float *weights, int64_t weights_stride, const int32_t *context_lens,
                                    int max_context_len, int num_seqs, int num_kv_heads, int budget, int sinks,
                                    int recent, float *weights_out, int32_t *kept, int32_t *kept_lens,
                                    void *stream) {
    if (num_seqs < 0 || num_seqs > 65535 || num_kv_heads <= 0 || max_context_len < 0 || budget <= 0 || sinks < 0 ||
        recent < 0 || static_cast<int64_t>(sinks) + recent > budget || weights_stride < max_context_len)
        return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    const auto bad = [](const void *q) { return !q || (reinterpret_cast<uintptr_t>(q) & 3u); };
    if (bad(weights) || bad(context_lens) || bad(kept) || bad(kept_lens) ||
        (reinterpret_cast<uintptr_t>(weights_out) & 3u))
        return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    SelectParams p{};
    p.weights = weights;
    p.weights_out = weights_out;
    p.context_lens = context_lens;
    p.kept = kept;
    p.kept_lens = kept_lens;
    p.status = status;
    p.weights_stride = weights_stride;
    p.len_cap = max_context_len;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    p.num_kv_heads = num_kv_heads;
    const dim3 grid(static_cast<unsigned>(num_kv_heads), static_cast<unsigned>(num_seqs));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (max_context_len <= 1024) evict_select_kernel<256, 4><<<grid, 256, 0, s>>>(p);
    else if (max_context_len <= 8192) evict_select_kernel<512, 16><<<grid, 512, 0, s>>>(p);
    else evict_select_kernel<1024, 32><<<grid, 1024, 0, s>>>(p);
    pkv::count_launch();
    return pkv::launch_status();
}

PKV_API pkv_status pkv_evict_compact(void *k_cache, void *v_cache, int64_t num_blocks, int64_t block_stride_elems,
                                     int num_kv_heads, int head_dim, int block_size, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                                     const int32_t *kept, const int32_t *kept_lens, int budget,
                                     const int32_t *dst_block_tables, int dst_max_blocks_per_seq, pkv_dtype dtype,
                                     void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16 && dtype != PKV_INT8) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_seqs > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || budget <= 0 || (dst_block_tables && dst_max_blocks_per_seq <= 0))
        return PKV_ERR_INVALID_ARG;
    const int elem_bytes = dtype == PKV_INT8 ? 1 : 2;
    const int64_t half_elems = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_elems < half_elems || (block_stride_elems * elem_bytes) % 16) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    const auto bad = [](const void *q) { return !q || (reinterpret_cast<uintptr_t>(q) & 3u); };
    if (bad(block_tables) || bad(context_lens) || bad(kept) || bad(kept_lens) ||
        (reinterpret_cast<uintptr_t>(dst_block_tables) & 3u))
        return PKV_ERR_INVALID_ARG;
    const bool in_place = !dst_block_tables || dst_block_tables == block_tables;
    if (in_place && dst_block_tables && dst_max_blocks_per_seq != max_blocks_per_seq) return PKV_ERR_INVALID_ARG;
    const auto capacity = [&](int64_t blocks) {
        return static_cast<int>(std::min<int64_t>(blocks * block_size, 0x7fffffff));
    };
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    CompactParams p{};
    p.k_cache = static_cast<char *>(k_cache);
    p.v_cache = static_cast<char *>(v_cache);
    p.src_tables = block_tables;
    p.dst_tables = in_place ? block_tables : dst_block_tables;
    p.context_lens = context_lens;
    p.kept = kept;
    p.kept_lens = kept_lens;
    p.status = status;
    p.num_blocks = num_blocks;
    p.block_stride = block_stride_elems * elem_bytes;
    p.src_stride = max_blocks_per_seq;
    p.dst_stride = in_place ? max_blocks_per_seq : dst_max_blocks_per_seq;
    p.budget = budget;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.src_cap = capacity(max_blocks_per_seq);
    p.dst_cap = capacity(p.dst_stride);
    const int max_kept = std::min(budget, std::min(p.src_cap, p.dst_cap));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int row_vecs = head_dim * elem_bytes / 16;
    if (row_vecs == 16) launch_compact<16>(p, in_place, max_kept, num_seqs, s);
    else if (row_vecs == 8) launch_compact<8>(p, in_place, max_kept, num_seqs, s);
    else launch_compact<4>(p, in_place, max_kept, num_seqs, s);
    pkv::count_launch();
    return pkv::launch_status();
}

}  // extern "C"
