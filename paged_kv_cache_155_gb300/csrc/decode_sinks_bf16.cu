// decode_sinks_bf16.cu -- bf16 instantiations of the paged decode kernels with a window and first tokens.
#include "decode_launch.cuh"

namespace pkv {
pkv_status launch_sinks_bf16(const DecodeParams &p, const DecodeMaps &m, int head_dim, int block_size, int gh, dim3 grid,
                           int merge_rows, cudaStream_t s) {
    return launch_decode_typed<__nv_bfloat16, __nv_bfloat16, true, true>(p, m, head_dim, block_size, gh, grid, merge_rows, s);
}
}  // namespace pkv
