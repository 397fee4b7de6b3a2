// decode_int4_bf16.cu -- bf16 instantiations of the 4-bit cache's decode kernels.
#include "decode_int4_launch.cuh"

namespace pkv {
pkv_status launch_int4_bf16(const DecodeParams &p, int head_dim, int block_size, int tiles, dim3 grid, int merge_rows,
                           cudaStream_t s) {
    return launch_int4_typed<__nv_bfloat16>(p, head_dim, block_size, tiles, grid, merge_rows, s);
}
}  // namespace pkv
