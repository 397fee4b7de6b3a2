// decode_int4_launch.cuh -- host-side dispatch to the 4-bit decode's instantiations of one
// element type (decode_int4_f16.cu, decode_int4_bf16.cu).
#pragma once

#include <atomic>

#include "decode_int4_kernel.cuh"
#include "pkv_host.h"

namespace pkv {

template <typename T, int D, int BS, int NT>
pkv_status launch_int4_one(const DecodeParams &p, dim3 grid, cudaStream_t stream) {
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
    if (launch_kernel(paged_decode_int4_kernel<T, D, BS, NT>, grid, dim3(G::kWarps * 32), G::kSmemBytes, stream, false,
                      p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

template <typename T, int D, int NT>
pkv_status launch_int4_bs(const DecodeParams &p, int block_size, dim3 grid, cudaStream_t s) {
    switch (block_size) {
        case 8: return launch_int4_one<T, D, 8, NT>(p, grid, s);
        case 16: return launch_int4_one<T, D, 16, NT>(p, grid, s);
        case 32: return launch_int4_one<T, D, 32, NT>(p, grid, s);
    }
    return PKV_ERR_UNSUPPORTED;
}

// tiles: column tiles of eight heads per block (1 or 2); merge_rows > 0: the merge follows.
template <typename T>
pkv_status launch_int4_typed(const DecodeParams &p, int head_dim, int block_size, int tiles, dim3 grid, int merge_rows,
                             cudaStream_t s) {
    pkv_status st;
    if (head_dim == 128)
        st = tiles == 1 ? launch_int4_bs<T, 128, 1>(p, block_size, grid, s) : launch_int4_bs<T, 128, 2>(p, block_size, grid, s);
    else
        st = tiles == 1 ? launch_int4_bs<T, 64, 1>(p, block_size, grid, s) : launch_int4_bs<T, 64, 2>(p, block_size, grid, s);
    if (st != PKV_OK || merge_rows == 0) return st;
    const bool wide = p.num_partitions >= kMergeWideFrom;
    const dim3 blocks(static_cast<unsigned>(wide ? merge_rows : (merge_rows + 3) / 4));
    auto merge = head_dim == 128 ? (wide ? paged_decode_merge_kernel<T, 128, 4> : paged_decode_merge_kernel<T, 128, 1>)
                                 : (wide ? paged_decode_merge_kernel<T, 64, 4> : paged_decode_merge_kernel<T, 64, 1>);
    if (launch_kernel(merge, blocks, dim3(128), 0, s, true, p, merge_rows) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    count_launch();
    return launch_status();
}

pkv_status launch_int4_f16(const DecodeParams &p, int head_dim, int block_size, int tiles, dim3 grid, int merge_rows,
                           cudaStream_t s);
pkv_status launch_int4_bf16(const DecodeParams &p, int head_dim, int block_size, int tiles, dim3 grid, int merge_rows,
                            cudaStream_t s);

}  // namespace pkv
