// tree_f16.cu -- fp16 instantiations of the drafted tree's attention kernels.
#include "prefill_launch.cuh"

namespace pkv {
pkv_status launch_tree_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &to, int block_size, int grid, cudaStream_t s) {
    return launch_tree<__half>(p, tq, tk, tv, to, block_size, grid, s);
}
}  // namespace pkv
