// decode_scored_i8.cu -- INT8-cache instantiations of the scored paged decode kernels
// (capped and biased scores, windows, weights).
#include "decode_launch.cuh"

namespace pkv {
pkv_status launch_scored_i8_f16(const DecodeParams &p, const DecodeMaps &m, int head_dim, int block_size, int gh,
                             dim3 grid, int merge_rows, cudaStream_t s, const WeightParams &w) {
    return launch_decode_typed<__half, int8_t, true>(p, m, head_dim, block_size, gh, grid, merge_rows, s, w);
}
pkv_status launch_scored_i8_bf16(const DecodeParams &p, const DecodeMaps &m, int head_dim, int block_size, int gh,
                             dim3 grid, int merge_rows, cudaStream_t s, const WeightParams &w) {
    return launch_decode_typed<__nv_bfloat16, int8_t, true>(p, m, head_dim, block_size, gh, grid, merge_rows, s, w);
}
}  // namespace pkv
