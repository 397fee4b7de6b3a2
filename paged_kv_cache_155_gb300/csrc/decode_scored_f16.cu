// decode_scored_f16.cu -- fp16 instantiations of the scored paged decode kernels
// (capped and biased scores, windows, weights).
#include "decode_launch.cuh"

namespace pkv {
pkv_status launch_scored_f16(const DecodeParams &p, const DecodeMaps &m, int head_dim, int block_size, int gh,
                             dim3 grid, int merge_rows, cudaStream_t s, const WeightParams &w) {
    return launch_decode_typed<__half, __half, true>(p, m, head_dim, block_size, gh, grid, merge_rows, s, w);
}
}  // namespace pkv
