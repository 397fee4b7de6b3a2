// prefill_launch.cuh -- host-side dispatch to the prefill kernel instantiations of one
// element type, plain or scored.
#pragma once

#include <atomic>

#include "prefill_tc_kernel.cuh"
#include "pkv_host.h"

namespace pkv {

template <typename T, int BS, int ORDER, int kForm>
pkv_status launch_prefill_one(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const CUtensorMap &to, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> configured_devices{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(configured_devices.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(paged_prefill_tc_kernel<T, BS, ORDER, kForm>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PrefillLayout::kSmemBytes) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_devices.fetch_or(bit, std::memory_order_acq_rel);
    }
    // planned order: placed while the plan kernel before it still runs
    if (launch_kernel(paged_prefill_tc_kernel<T, BS, ORDER, kForm>, dim3(grid), dim3(PrefillLayout::kThreads),
                      PrefillLayout::kSmemBytes, stream, ORDER == kOrderPlanned || kForm == kTreeForm, tq, tk, tv, to, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

template <typename T, int BS, bool kScored>
pkv_status launch_prefill_bs(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                             const CUtensorMap &tv, const CUtensorMap &to, int grid, cudaStream_t s) {
    if constexpr (kScored) {
        if constexpr (!std::is_same<T, __half>::value) {
            if (p.fixed_ref)
                return p.order == kOrderPlanned ? launch_prefill_one<T, BS, kOrderPlanned, kFixedForm>(p, tq, tk, tv, to, grid, s)
                                                : launch_prefill_one<T, BS, kOrderRowTiles, kFixedForm>(p, tq, tk, tv, to, grid, s);
        }
        if (p.cap_out == 0.f)
            return p.order == kOrderPlanned ? launch_prefill_one<T, BS, kOrderPlanned, kUncappedForm>(p, tq, tk, tv, to, grid, s)
                                            : launch_prefill_one<T, BS, kOrderRowTiles, kUncappedForm>(p, tq, tk, tv, to, grid, s);
        return p.order == kOrderPlanned ? launch_prefill_one<T, BS, kOrderPlanned, kScoredForm>(p, tq, tk, tv, to, grid, s)
                                        : launch_prefill_one<T, BS, kOrderRowTiles, kScoredForm>(p, tq, tk, tv, to, grid, s);
    }
    else if (p.order == kOrderSortedGroups)
        return launch_prefill_one<T, BS, kOrderSortedGroups, kPlainForm>(p, tq, tk, tv, to, grid, s);
    else if (p.order == kOrderPairs) return launch_prefill_one<T, BS, kOrderPairs, kPlainForm>(p, tq, tk, tv, to, grid, s);
    else return launch_prefill_one<T, BS, kOrderRowTiles, kPlainForm>(p, tq, tk, tv, to, grid, s);
}

template <typename T, bool kScored = false>
pkv_status launch_prefill(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                          int max_query_len, cudaStream_t s) {
    pkv_status st = PKV_ERR_UNSUPPORTED;
    if (block_size == 8) st = launch_prefill_bs<T, 8, kScored>(p, tq, tk, tv, to, grid, s);
    else if (block_size == 16) st = launch_prefill_bs<T, 16, kScored>(p, tq, tk, tv, to, grid, s);
    else if (block_size == 32) st = launch_prefill_bs<T, 32, kScored>(p, tq, tk, tv, to, grid, s);
    if (st != PKV_OK || p.splits == 1) return st;
    const int64_t rows = static_cast<int64_t>(max_query_len) * p.num_q_heads;
    const dim3 mgrid(static_cast<unsigned>((rows + 3) / 4), static_cast<unsigned>(p.num_seqs));
    paged_prefill_merge_kernel<T, kScored><<<mgrid, 128, 0, s>>>(p);
    count_launch();
    return launch_status();
}

// The sink form (a window and first tokens): planned items, or row tiles when the KV ranges are split.
template <typename T>
pkv_status launch_prefill_sinks(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                int max_query_len, cudaStream_t s) {
    auto launch = [&](auto bs) -> pkv_status {
        constexpr int BS = decltype(bs)::value;
        return p.order == kOrderPlanned ? launch_prefill_one<T, BS, kOrderPlanned, kSinkForm>(p, tq, tk, tv, to, grid, s)
                                        : launch_prefill_one<T, BS, kOrderRowTiles, kSinkForm>(p, tq, tk, tv, to, grid, s);
    };
    const pkv_status st = block_size == 8    ? launch(std::integral_constant<int, 8>{})
                          : block_size == 16 ? launch(std::integral_constant<int, 16>{})
                                             : launch(std::integral_constant<int, 32>{});
    if (st != PKV_OK || p.splits == 1) return st;
    const int64_t rows = static_cast<int64_t>(max_query_len) * p.num_q_heads;
    const dim3 mgrid(static_cast<unsigned>((rows + 3) / 4), static_cast<unsigned>(p.num_seqs));
    paged_prefill_merge_kernel<T, true, true><<<mgrid, 128, 0, s>>>(p);
    count_launch();
    return launch_status();
}

// The tree form: the stream order over all SMs, then the merge of the units that it cut.
template <typename T>
pkv_status launch_tree(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                       const CUtensorMap &to, int block_size, int grid, cudaStream_t s) {
    const pkv_status st =
        block_size == 8    ? launch_prefill_one<T, 8, kOrderStream, kTreeForm>(p, tq, tk, tv, to, grid, s)
        : block_size == 16 ? launch_prefill_one<T, 16, kOrderStream, kTreeForm>(p, tq, tk, tv, to, grid, s)
                           : launch_prefill_one<T, 32, kOrderStream, kTreeForm>(p, tq, tk, tv, to, grid, s);
    if (st != PKV_OK) return st;
    const int entries = p.by_unit ? p.num_seqs * p.num_kv_heads * p.row_tiles : grid;
    const bool shared = p.by_unit && entries * 8 <= grid;  // units cut into eight pieces or more
    if (launch_kernel(shared ? paged_tree_merge_kernel<T, 4> : paged_tree_merge_kernel<T, 1>, dim3(static_cast<unsigned>(entries), 16),
                      dim3(shared ? 512 : 128), 0, s, true, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

// Defined in prefill_scored_f16.cu / prefill_scored_bf16.cu.
pkv_status launch_prefill_scored_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                     const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                     int max_query_len, cudaStream_t s);
pkv_status launch_prefill_scored_bf16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                      const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                      int max_query_len, cudaStream_t s);

// Defined in prefill_sinks_f16.cu / _bf16.cu and tree_f16.cu / _bf16.cu.
pkv_status launch_prefill_sinks_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                    const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                    int max_query_len, cudaStream_t s);
pkv_status launch_prefill_sinks_bf16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                     const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                     int max_query_len, cudaStream_t s);
pkv_status launch_tree_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const CUtensorMap &to, int block_size, int grid, cudaStream_t s);
pkv_status launch_tree_bf16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &to, int block_size, int grid, cudaStream_t s);

}  // namespace pkv
