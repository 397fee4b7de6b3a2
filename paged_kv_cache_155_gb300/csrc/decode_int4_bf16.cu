// decode_int4_bf16.cu -- bf16 instantiations of the 4-bit cache's decode kernels.
#include "decode_int4_launch.cuh"

namespace pkv {
pkv_status launch_int4_bf16(const Int4Params &p, int head_dim, int block_size, int heads_per_block, int grid, cudaStream_t s) {
    return launch_int4_typed<__nv_bfloat16>(p, head_dim, block_size, heads_per_block, grid, s);
}
}  // namespace pkv
