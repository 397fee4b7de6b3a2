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
    int vectors;           // rows of weights start 16-byte aligned
};

// CL CTAs (a cluster) per (KV head, sequence).  The kept tokens are the first `sinks`,
// the last `recent` and, of those between, the `need` heaviest, equal weights by lower
// index.  The threshold -- the need-th largest key -- is found from the top, 11, 11 and
// 10 bits at a time: count the keys that share the bits found so far by their next
// digit in shared memory, find the digit at which the count from above passes `need`,
// and descend; done as soon as the keys from some digit on are exactly `need`.  In a
// cluster every CTA counts its share and reads the others' counts.  A row's tokens go
// in batches of CL x EB x THREADS, CTA after CTA, EB consecutive ones per thread; the
// first HELD batches stay in registers, a longer row's others are read again (from L2)
// in each pass.  The kept positions then leave in ascending order, batch by batch, by
// one prefix count of the threads over the block and the cluster, gathered in shared
// memory so that the stores are whole lines.
//
// Bound by the latency of its passes, not by bytes (4 read and 4 written per token).
// Measured: 256 rows of 2048-4096 tokens 11 us (24 us when the threshold came from
// repeated counting against bisecting candidates), 24 rows of 32768 18 us with clusters
// of eight (31 us with one CTA a row, which 24 SMs then work on alone), 512 rows of 32768
// 80 us (130 us with strided tokens, a ballot per 32 of them and stores straight to the
// row).
template <int THREADS, int EB, int HELD, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const SelectParams p) {
    constexpr int WARPS = THREADS / 32, PART = EB * THREADS, BATCH = CL * PART;
    constexpr int BINS = 2048, PER_BIN = BINS / THREADS;
    constexpr int COUNTS = CL > 1 ? 2 * BINS : BINS;
    static_assert(BINS % THREADS == 0 && WARPS <= 32 && EB % 4 == 0 && PART < 65536, "whole bins per thread, counts of 16 bits");
    // the threshold's counts, then a batch's kept positions and their weights
    __shared__ uint32_t shared[COUNTS > 2 * PART ? COUNTS : 2 * PART];
    uint32_t *const bins = shared, *const sums = shared + (CL > 1 ? BINS : 0);  // sums: the bins over the cluster
    __shared__ uint32_t warp_sum[WARPS];
    __shared__ uint32_t found[3];       // the digit, the keys above it, the keys in it
    __shared__ uint32_t totals[2][CL];  // (kept outright, ties) of each CTA's part of a batch, 16 bits each
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
    // a thread's EB tokens of a batch, from first_of on
    const auto first_of = [&](int batch) { return batch * BATCH + rank * PART + tid * EB; };
    const auto load = [&](int batch, float (&v)[EB]) {
        const int t0 = first_of(batch);
        if (p.vectors && t0 + EB <= len) {
#pragma unroll
            for (int e = 0; e < EB; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(w + t0 + e);
                v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < EB; ++e) v[e] = t0 + e < len ? w[t0 + e] : 0.f;
        }
    };
    const auto below = [](int n) { return (1u << max(0, min(n, EB))) - 1u; };  // the lowest n of EB bits
    float val[HELD][EB];
#pragma unroll
    for (int b = 0; b < HELD; ++b) load(b, val[b]);
    for (int i = keep + rtid; i < p.budget; i += CL * THREADS) kept[i] = -1;
    // the tokens [mid0, mid1) compete for `need` places, the others stay
    const bool all = len <= p.budget;
    const uint32_t need = all ? 0u : static_cast<uint32_t>(p.budget - p.sinks - p.recent);
    const int mid0 = all ? 0 : p.sinks, mid1 = all ? 0 : len - p.recent;
    const auto competing = [&](int batch) {
        const int t0 = first_of(batch);
        return below(mid1 - t0) & ~below(mid0 - t0);
    };

    // the keys >= thr stay, or (not exact) those > thr and the first `ties` that equal it
    uint32_t thr = 0xffffffffu, ties = 0u;  // (need 0: no key is that large)
    bool exact = true;
    if (need > 0) {
        thr = 0u;
        exact = false;
        uint32_t left = need;  // of the keys that share thr's digits so far
        // digits: bits 31..21, 20..10, 9..0
        for (int shift = 21, width = 11; width > 0 && !exact; width = shift == 21 ? 11 : shift == 10 ? 10 : 0,
                 shift = shift == 21 ? 10 : 0) {
            for (int i = tid; i < BINS; i += THREADS) bins[i] = 0u;
            __syncthreads();
            const uint32_t mask = (1u << width) - 1u;
            const auto count = [&](int batch, const float (&v)[EB]) {
                const uint32_t comp = competing(batch);
#pragma unroll
                for (int e = 0; e < EB; ++e) {
                    const uint32_t k = weight_key(v[e]);
                    // the digits above are thr's (all of a key's, in the first pass)
                    if (((comp >> e) & 1u) && (shift == 21 || (k >> (shift + width)) == (thr >> (shift + width))))
                        atomicAdd(&bins[(k >> shift) & mask], 1u);
                }
            };
#pragma unroll
            for (int b = 0; b < HELD; ++b) count(b, val[b]);
            for (int b = HELD; b * BATCH < mid1; ++b) {
                float v[EB];
                load(b, v);
                count(b, v);
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
                mine[i] = sums[BINS - 1 - (tid * PER_BIN + i)];
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
    // what stays outright has a key from `from` on (no weight has the key 2^32 - 1)
    const uint32_t from = exact ? thr : thr + 1u;

    if (CL > 1 && need == 0) sync_row();  // the other CTAs run, and so can be stored to
    uint32_t *const out_pos = shared, *const out_weight = shared + PART;
    uint32_t done = 0u, ties_done = 0u;  // tokens kept outright / equal to the threshold, before this batch
    const auto emit = [&](int b, const float (&v)[EB]) {
        const int t0 = first_of(b);
        const uint32_t comp = competing(b);
        uint32_t in = below(len - t0) & ~comp, tie = 0u;
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const uint32_t k = weight_key(v[e]);
            in |= static_cast<uint32_t>(k >= from) << e & comp;
            tie |= static_cast<uint32_t>(k == thr) << e & comp;
        }
        if (exact) tie = 0u;
        // (outright, ties) before this thread's tokens: each half of a sum stays below 2^16
        const uint32_t own = __popc(in) | (__popc(tie) << 16);
        uint32_t incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        const uint32_t ws = lane < WARPS ? warp_sum[lane] : 0u;
        const uint32_t before = incl - own + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u);
        const uint32_t part = __reduce_add_sync(0xffffffffu, ws);
        // (two sets of totals in turn: a CTA may be a batch ahead, never two)
        if constexpr (CL > 1) {
            if (tid < CL) store_remote(remote(pkv::smem_addr(&totals[b & 1][rank]), tid), part);
        }
        // every weight of this batch is in registers behind this barrier, and ranks only
        // move tokens down: weights_out may be weights
        sync_row();
        uint32_t in_base = done, tie_base = ties_done;  // before this CTA's part
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            const uint32_t n = CL > 1 ? totals[b & 1][c] : part;
            if (c < rank) {
                in_base += n & 0xffffu;
                tie_base += n >> 16;
            }
            done += n & 0xffffu;
            ties_done += n >> 16;
        }
        const uint32_t ties_out = min(tie_base, ties);  // of the ties before the part, those that stay
        const uint32_t base = in_base + ties_out;
        const uint32_t kept_here = (part & 0xffffu) + min(tie_base + (part >> 16), ties) - ties_out;
        uint32_t tie_at = tie_base + (before >> 16);
        uint32_t at = (before & 0xffffu) + min(tie_at, ties) - ties_out;
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const bool is_tie = (tie >> e) & 1u;
            if (((in >> e) & 1u) || (is_tie && tie_at < ties)) {
                out_pos[at] = t0 + e;
                if (wout) out_weight[at] = __float_as_uint(v[e]);
                ++at;
            }
            tie_at += is_tie;
        }
        __syncthreads();
        for (uint32_t i = tid; i < kept_here; i += THREADS) {
            kept[base + i] = static_cast<int32_t>(out_pos[i]);
            if (wout) wout[base + i] = __uint_as_float(out_weight[i]);
        }
    };
#pragma unroll
    for (int b = 0; b < HELD; ++b)
        if (b * BATCH < len) emit(b, val[b]);
    for (int b = HELD; b * BATCH < len; ++b) {
        float v[EB];
        load(b, v);
        emit(b, v);
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
    int src_stride, dst_stride, budget, num_kv_heads, src_cap, dst_cap;
    int block_shift;  // log2 of the block size
};

constexpr int kMoveUnroll = 4;
// In place, a CTA's tiles follow one another: larger ones (the same 268 MB: 256 threads 61
// us, 512 58, 1024 74; 34 MB of four sequences 16.5 / 11.2 / 11.1).
__host__ __device__ constexpr int move_threads(bool in_place) { return in_place ? 512 : 128; }

// The bytes of token row (block, head, offset) of one pool half.
__device__ __forceinline__ int64_t row_offset(const CompactParams &p, int blk, int h, int t, int row_bytes) {
    return static_cast<int64_t>(blk) * p.block_stride +
           ((static_cast<int64_t>(h) << p.block_shift) + (t & ((1 << p.block_shift) - 1))) * row_bytes;
}

// Moves token row kept[i] to position i.  VECS 16-byte vectors of a row per CTA
// column group; grid: (tiles x column groups x 2 halves, KV head, sequence).
// Into fresh blocks (IN_PLACE false) the tiles are independent.  In place, a CTA
// walks its column group's tiles in ascending order: kept[i] >= i and kept ascends,
// so a tile's stores (positions [a, b)) can only meet rows that tiles up to this one
// read, never a later tile's sources -- one barrier between a tile's loads and its
// stores orders them, and column groups never meet.
// Bound by memory: rows of 256 bytes gathered at random, read and written once
// (plain loads and stores instead of streaming ones: 6% slower).  Measured into fresh
// blocks: 268 MB moved in 44 us, 6.0 TB/s, 0.89 of the copy rate of large contiguous
// arrays; eight or two rows per thread 52 / 49, 256 threads instead of 128 44.6, block
// offsets by division instead of shifts 50 (the kept rows' order hardly matters: adjacent
// ones 44).
template <int ROW_VECS, int VECS, bool IN_PLACE>
__global__ void __launch_bounds__(move_threads(IN_PLACE)) evict_compact_kernel(const CompactParams p) {
    constexpr int ROWS = move_threads(IN_PLACE) / VECS, TILE = ROWS * kMoveUnroll, GROUPS = ROW_VECS / VECS;
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
            const int sb = src_table[t >> p.block_shift], db = dst_table[i >> p.block_shift];
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
        return pkv::launch_kernel(evict_compact_kernel<ROW_VECS, VECS, true>, grid, dim3(move_threads(true)), 0, s, true, p);
    } else {
        constexpr int TILE = move_threads(false) / ROW_VECS * kMoveUnroll;
        const dim3 grid(2 * ((max_kept + TILE - 1) / TILE), p.num_kv_heads, num_seqs);
        return pkv::launch_kernel(evict_compact_kernel<ROW_VECS, ROW_VECS, false>, grid, dim3(move_threads(false)), 0, s, true, p);
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
    // one KV head's CTA writes a sequence's new length while the others' may still read the old one
    if (kept_lens < context_lens + num_seqs && context_lens < kept_lens + num_seqs) return PKV_ERR_INVALID_ARG;
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
    p.vectors = weights_stride % 4 == 0 && pkv::aligned16(weights);
    const dim3 grid(static_cast<unsigned>(num_kv_heads), static_cast<unsigned>(num_seqs));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Rows past 8192 tokens spread over a cluster as large as leaves every cluster resident
    // at once (two CTAs per SM): one CTA would work through the row on one SM, but a second
    // wave of clusters would wait for the first.  (Rows of 32768, this rule against always
    // eight: 72 rows 20 us / 34 us, 152 rows 29 / 61, 512 rows 80 / 191.)
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
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
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
