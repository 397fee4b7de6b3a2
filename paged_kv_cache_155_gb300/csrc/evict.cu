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

// Shared memory of the other CTAs of a cluster: the address that `addr` has in CTA
// `rank`, loads and stores there, and the barrier of the whole cluster (which also
// makes earlier stores visible).
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t load_remote(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMaxTokens = 1 << 30;  // of a context or a budget: indices a step past it still fit 32 bits

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

// CL CTAs (a cluster) per (KV head, sequence).  The kept tokens are the first `sinks`,
// the last `recent` and, of those between, the `need` heaviest, equal weights by lower
// index.  The threshold -- the need-th largest key -- is found from the top, 11, 11 and
// 10 bits at a time: count the keys that share the bits found so far by their next
// digit in shared memory, find the digit at which the count from above passes `need`,
// and descend; done as soon as the keys from some digit on are exactly `need`.  In a
// cluster every CTA counts its share and reads the others' counts.  A row's tokens go
// in batches of CL x EB x THREADS, CTA after CTA; the keys of the first HELD batches
// stay in registers, a longer row's others are read again (from L2) in each pass.  The
// kept positions then leave in ascending order, batch by batch, by a prefix count over
// the block and the cluster.
//
// Bound by the latency of its passes, not by bytes (4 read and 4 written per token).
// Measured: 256 rows of 2048-4096 tokens 12 us (24 us when the threshold came from
// repeated counting against bisecting candidates), 24 rows of 32768 19 us with clusters
// of eight (31 us with one CTA a row, which 24 SMs then work on alone).
template <int THREADS, int EB, int HELD, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(THREADS) evict_select_kernel(const SelectParams p) {
    constexpr int WARPS = THREADS / 32, PART = EB * THREADS, BATCH = CL * PART;
    constexpr int BINS = 2048, PER_BIN = BINS / THREADS;
    static_assert(BINS % THREADS == 0 && CL <= 32 && EB * HELD <= 32, "whole bins per thread, masks of 32 bits");
    __shared__ uint32_t bins[BINS];
    __shared__ uint32_t sums[CL > 1 ? BINS : 1];  // the bins summed over the cluster
    __shared__ uint32_t warp_sum[WARPS];
    __shared__ uint32_t found[3];            // the digit, the keys above it, the keys in it
    __shared__ uint32_t totals[EB * WARPS];  // (kept outright, ties) of each 32 tokens, 16 bits each
    __shared__ uint32_t bases[EB * WARPS];   // their exclusive prefix
    __shared__ uint32_t part_total;          // their sum
    const int rank = blockIdx.x % CL;
    const auto sync_row = [] {
        if constexpr (CL > 1) cluster_sync();
        else __syncthreads();
    };
    const int h = blockIdx.x / CL, seq = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = static_cast<int64_t>(seq) * p.num_kv_heads + h;
    int len = p.context_lens[seq];
    if (len < 0 || len > p.len_cap) {
        if (tid == 0 && blockIdx.x == 0) pkv::raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        len = len < 0 ? 0 : p.len_cap;
    }
    const int keep = min(len, p.budget);
    if (blockIdx.x == 0 && tid == 0) p.kept_lens[seq] = keep;
    const float *w = p.weights + row * p.weights_stride;
    float *wout = p.weights_out ? p.weights_out + row * p.weights_stride : nullptr;
    int32_t *kept = p.kept + row * p.budget;
    const int rtid = rank * THREADS + tid;  // thread of the row
    for (int i = keep + rtid; i < p.budget; i += CL * THREADS) kept[i] = -1;
    const bool all = len <= p.budget;
    const int mid0 = p.sinks, mid1 = len - p.recent;  // the tokens that compete, when !all
    const uint32_t need = all ? 0u : static_cast<uint32_t>(p.budget - p.sinks - p.recent);
    const auto token = [&](int batch, int e) { return batch * BATCH + rank * PART + e * THREADS + tid; };

    // the keys >= thr stay, or (not exact) those > thr and the first `ties` that equal it
    uint32_t thr = 0u, ties = 0u;
    bool exact = false;
    if (need > 0) {
        uint32_t key[EB * HELD];
        uint32_t held = 0u;  // bit i: key i's token competes
#pragma unroll
        for (int i = 0; i < EB * HELD; ++i) {
            const int t = token(i / EB, i % EB);
            const bool competes = t >= mid0 && t < mid1;
            key[i] = competes ? __float_as_uint(w[t]) : 0u;
            held |= static_cast<uint32_t>(competes) << i;
        }
#pragma unroll
        for (int i = 0; i < EB * HELD; ++i) key[i] = weight_key(__uint_as_float(key[i]));
        uint32_t left = need;  // of the keys that share thr's digits so far
        // digits: bits 31..21, 20..10, 9..0
        for (int shift = 21, width = 11; width > 0 && !exact; width = shift == 21 ? 11 : shift == 10 ? 10 : 0,
                 shift = shift == 21 ? 10 : 0) {
            for (int i = tid; i < BINS; i += THREADS) bins[i] = 0u;
            __syncthreads();
            const uint32_t mask = (1u << width) - 1u;
            auto count = [&](uint32_t k) {
                // the digits above are thr's (all of a key's, in the first pass)
                if (shift == 21 || (k >> (shift + width)) == (thr >> (shift + width)))
                    atomicAdd(&bins[(k >> shift) & mask], 1u);
            };
#pragma unroll
            for (int i = 0; i < EB * HELD; ++i)
                if ((held >> i) & 1u) count(key[i]);
            for (int b = HELD; b * BATCH < mid1; ++b)
                for (int e = 0; e < EB; ++e) {
                    const int t = token(b, e);
                    if (t >= mid0 && t < mid1) count(weight_key(w[t]));
                }
            sync_row();
            if constexpr (CL > 1) {
                // this CTA's share of the bins, summed over the cluster and sent to every CTA
                for (int i = tid; i < BINS / CL; i += THREADS) {
                    const uint32_t mine = pkv::smem_addr(&bins[rank * (BINS / CL) + i]);
                    const uint32_t sums_at = pkv::smem_addr(&sums[rank * (BINS / CL) + i]);
                    uint32_t n = 0u;
#pragma unroll
                    for (int c = 0; c < CL; ++c) n += load_remote(remote(mine, c));
#pragma unroll
                    for (int c = 0; c < CL; ++c) store_remote(remote(sums_at, c), n);
                }
                sync_row();
            }
            // thread i holds the PER_BIN bins from the top: keys above them by a block-wide prefix
            uint32_t mine[PER_BIN], sum = 0u;
#pragma unroll
            for (int i = 0; i < PER_BIN; ++i) {
                const int at = BINS - 1 - (tid * PER_BIN + i);
                mine[i] = CL > 1 ? sums[at] : bins[at];
                sum += mine[i];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            uint32_t above = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
#pragma unroll
            for (int i = 0; i < PER_BIN; ++i) {
                if (above < left && above + mine[i] >= left) {  // one bin of one thread
                    found[0] = BINS - 1 - (tid * PER_BIN + i);
                    found[1] = above;
                    found[2] = mine[i];
                }
                above += mine[i];
            }
            __syncthreads();
            thr |= found[0] << shift;
            left -= found[1];
            exact = found[2] == left;  // every key from this digit on stays
        }
        ties = exact ? 0u : left;
    }

    uint32_t done = 0u, ties_done = 0u;  // tokens kept outright / equal to the threshold, before this batch
    for (int b = 0; b * BATCH < len; ++b) {
        float val[EB];
#pragma unroll
        for (int e = 0; e < EB; ++e) val[e] = token(b, e) < len ? w[token(b, e)] : 0.f;
        uint32_t in_mask[EB], tie_mask[EB];  // the warp's tokens e: stays outright / equals the threshold
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int t = token(b, e);
            const uint32_t k = weight_key(val[e]);
            const bool fixed = t < len && (all || t < mid0 || t >= mid1);
            const bool competes = need > 0 && t >= mid0 && t < mid1;
            in_mask[e] = __ballot_sync(0xffffffffu, fixed || (competes && (exact ? k >= thr : k > thr)));
            tie_mask[e] = __ballot_sync(0xffffffffu, competes && !exact && k == thr);
            if (lane == 0) totals[e * WARPS + warp] = __popc(in_mask[e]) | (__popc(tie_mask[e]) << 16);
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
            if (lane == 31) part_total = incl;
        }
        // every weight of this batch is in registers behind this barrier, and ranks only
        // move tokens down: weights_out may be weights
        sync_row();
        uint32_t in_base = done, tie_base = ties_done;
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            const uint32_t v = CL > 1 ? load_remote(remote(pkv::smem_addr(&part_total), c)) : part_total;
            if (c < rank) {
                in_base += v & 0xffffu;
                tie_base += v >> 16;
            }
            done += v & 0xffffu;
            ties_done += v >> 16;
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const uint32_t before = bases[e * WARPS + warp], mask = (1u << lane) - 1u;
            const uint32_t in_before = in_base + (before & 0xffffu) + __popc(in_mask[e] & mask);
            const uint32_t tie_before = tie_base + (before >> 16) + __popc(tie_mask[e] & mask);
            if (((in_mask[e] >> lane) & 1u) || (((tie_mask[e] >> lane) & 1u) && tie_before < ties)) {
                const uint32_t rank_of = in_before + min(tie_before, ties);
                kept[rank_of] = token(b, e);
                if (wout) wout[rank_of] = val[e];
            }
        }
        sync_row();  // before the shared counts change, or a CTA whose counts are read exits
    }
    if (wout)
        for (int i = keep + rtid; i < len; i += CL * THREADS) wout[i] = 0.f;  // slots the next tokens take
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
// Bound by memory: rows of 256 bytes gathered at random, read and written once
// (streaming loads and stores: 50 us, plain ones 53).  Measured into fresh blocks: 268 MB
// moved in 50 us, 5.3 TB/s, 0.79 of the copy rate of large contiguous arrays; eight, two
// or one row per thread and the heads fastest in the grid: 60 / 51 / 57 / 50.
template <int ROW_VECS, int VECS, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
    constexpr int ROWS = kMoveThreads / VECS, TILE = ROWS * kMoveUnroll, GROUPS = ROW_VECS / VECS;
    pkv::pdl_wait();  // launched ahead of the kernel before it (the choice of what to keep)
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
            x[u] = __ldcs(reinterpret_cast<const uint4 *>(base + row_offset(p, sb, h, t, ROW_VECS * 16) + col));
            to[u] = row_offset(p, db, h, i, ROW_VECS * 16) + col;
        }
        if (IN_PLACE) __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (to[u] >= 0) __stcs(reinterpret_cast<uint4 *>(base + to[u]), x[u]);
        if (!IN_PLACE) break;
    }
}

template <int ROW_VECS>
cudaError_t launch_compact(const CompactParams &p, bool in_place, int max_kept, int num_seqs, cudaStream_t s) {
    if (in_place) {
        constexpr int VECS = ROW_VECS < 4 ? ROW_VECS : 4;  // 64-byte columns: more chains, whole sectors
        const dim3 grid(2 * (ROW_VECS / VECS), p.num_kv_heads, num_seqs);
        return pkv::launch_kernel(evict_compact_kernel<ROW_VECS, VECS, true>, grid, dim3(kMoveThreads), 0, s, true, p);
    } else {
        constexpr int TILE = kMoveThreads / ROW_VECS * kMoveUnroll;
        const dim3 grid(2 * ((max_kept + TILE - 1) / TILE), p.num_kv_heads, num_seqs);
        return pkv::launch_kernel(evict_compact_kernel<ROW_VECS, ROW_VECS, false>, grid, dim3(kMoveThreads), 0, s, true, p);
    }
}

}  // namespace

extern "C" {

PKV_API pkv_status pkv_evict_select(const float *weights, int64_t weights_stride, const int32_t *context_lens,
                                    int max_context_len, int num_seqs, int num_kv_heads, int budget, int sinks,
                                    int recent, float *weights_out, int32_t *kept, int32_t *kept_lens,
                                    void *stream) {
    if (num_seqs < 0 || num_seqs > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 || max_context_len < 0 || budget <= 0 || sinks < 0 ||
        recent < 0 || static_cast<int64_t>(sinks) + recent > budget || weights_stride < max_context_len ||
        max_context_len > kMaxTokens || budget > kMaxTokens)
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
    // Rows past 8192 tokens spread over a cluster as large as leaves every cluster resident
    // at once (two CTAs per SM): one CTA would work through the row on one SM, but a second
    // wave of clusters would wait for the first.  (Rows of 32768, this rule against always
    // eight: 72 rows 25 us / 36 us, 152 rows 45 / 73, 512 rows 130 / 223.)
    if (max_context_len <= 1024) {
        evict_select_kernel<256, 4, 1, 1><<<grid, 256, 0, s>>>(p);
    } else if (max_context_len <= 8192) {
        evict_select_kernel<512, 8, 2, 1><<<grid, 512, 0, s>>>(p);
    } else {
        const int sms = pkv::current_sm_count();
        if (sms <= 0) return PKV_ERR_CUDA;
        const int64_t rows = static_cast<int64_t>(num_kv_heads) * num_seqs, slots = 2LL * sms;
        if (rows * 8 <= slots) evict_select_kernel<512, 8, 2, 8><<<dim3(grid.x * 8, grid.y), 512, 0, s>>>(p);
        else if (rows * 4 <= slots) evict_select_kernel<512, 8, 2, 4><<<dim3(grid.x * 4, grid.y), 512, 0, s>>>(p);
        else if (rows * 2 <= slots) evict_select_kernel<512, 8, 2, 2><<<dim3(grid.x * 2, grid.y), 512, 0, s>>>(p);
        else evict_select_kernel<512, 8, 2, 1><<<grid, 512, 0, s>>>(p);
    }
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
        max_blocks_per_seq <= 0 || budget <= 0 || budget > kMaxTokens || (dst_block_tables && dst_max_blocks_per_seq <= 0))
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
    const cudaError_t err = row_vecs == 16  ? launch_compact<16>(p, in_place, max_kept, num_seqs, s)
                            : row_vecs == 8 ? launch_compact<8>(p, in_place, max_kept, num_seqs, s)
                                            : launch_compact<4>(p, in_place, max_kept, num_seqs, s);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    pkv::count_launch();
    return pkv::launch_status();
}

}  // extern "C"
