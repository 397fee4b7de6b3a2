// decode_int4_launch.cuh -- host-side dispatch to the 4-bit decode's instantiations of one
// element type (decode_int4_f16.cu, decode_int4_bf16.cu).
#pragma once

#include <algorithm>
#include <atomic>

#include "decode_int4_kernel.cuh"
#include "pkv_host.h"

namespace pkv {

template <typename T, int D, int BS, int NT>
pkv_status launch_int4_one(const Int4Params &p, int grid, cudaStream_t stream) {
    using G = DecodeInt4Geom<D, BS, NT>;
    static std::atomic<uint64_t> configured_devices{0};  // bit per device ordinal
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(configured_devices.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(paged_decode_int4_kernel<T, D, BS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 G::kSmemBytes) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_devices.fetch_or(bit, std::memory_order_acq_rel);
    }
    if (launch_kernel(paged_decode_int4_kernel<T, D, BS, NT>, dim3(static_cast<unsigned>(grid)), dim3(G::kWarps * 32), G::kSmemBytes, stream, true,
                      p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

template <typename T, int D, int NT>
pkv_status launch_int4_bs(const Int4Params &p, int block_size, int grid, cudaStream_t s) {
    switch (block_size) {
        case 8: return launch_int4_one<T, D, 8, NT>(p, grid, s);
        case 16: return launch_int4_one<T, D, 16, NT>(p, grid, s);
        case 32: return launch_int4_one<T, D, 32, NT>(p, grid, s);
    }
    return PKV_ERR_UNSUPPORTED;
}

// heads per block: 4 (paired), 8 or 16 (one or two column tiles); grid CTAs, then the merge of the units that
// their workers cut.
template <typename T>
pkv_status launch_int4_typed(const Int4Params &p, int head_dim, int block_size, int heads_per_block, int grid, cudaStream_t s) {
    pkv_status st;
    if (head_dim == 128)
        st = heads_per_block == 4   ? launch_int4_bs<T, 128, 0>(p, block_size, grid, s)
             : heads_per_block == 8 ? launch_int4_bs<T, 128, 1>(p, block_size, grid, s)
                                    : launch_int4_bs<T, 128, 2>(p, block_size, grid, s);
    else
        st = heads_per_block == 4   ? launch_int4_bs<T, 64, 0>(p, block_size, grid, s)
             : heads_per_block == 8 ? launch_int4_bs<T, 64, 1>(p, block_size, grid, s)
                                    : launch_int4_bs<T, 64, 2>(p, block_size, grid, s);
    if (st != PKV_OK) return st;
    // units cut into many pieces: four warps share a head's
    const int64_t units = static_cast<int64_t>(p.num_seqs) * p.units;
    const bool shared = p.by_unit && grid * 4 >= 16 * units;
    auto merge = head_dim == 128 ? (shared ? paged_decode_int4_merge_kernel<T, 128, 4> : paged_decode_int4_merge_kernel<T, 128, 1>)
                                 : (shared ? paged_decode_int4_merge_kernel<T, 64, 4> : paged_decode_int4_merge_kernel<T, 64, 1>);
    const int heads = std::min(p.group, heads_per_block);
    const dim3 blocks(static_cast<unsigned>(p.by_unit ? units : grid * 4),
                      static_cast<unsigned>(shared ? heads : p.by_unit ? (heads + 3) / 4 : 1));
    if (launch_kernel(merge, blocks, dim3(128), 0, s, true, p, heads_per_block) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

pkv_status launch_int4_f16(const Int4Params &p, int head_dim, int block_size, int heads_per_block, int grid, cudaStream_t s);
pkv_status launch_int4_bf16(const Int4Params &p, int head_dim, int block_size, int heads_per_block, int grid, cudaStream_t s);

}  // namespace pkv
