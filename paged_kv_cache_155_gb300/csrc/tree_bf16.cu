// tree_bf16.cu -- bf16 instantiations of the drafted tree's attention kernels.
#include "prefill_launch.cuh"

namespace pkv {
pkv_status launch_tree_bf16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &to, int block_size, int grid, cudaStream_t s) {
    return launch_tree<__nv_bfloat16>(p, tq, tk, tv, to, block_size, grid, s);
}
}  // namespace pkv
