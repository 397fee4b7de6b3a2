// prefill_sinks_f16.cu -- fp16 instantiations of the prefill kernels with a window and first tokens.
#include "prefill_launch.cuh"

namespace pkv {
pkv_status launch_prefill_sinks_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                     const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                     int max_query_len, cudaStream_t s) {
    return launch_prefill_sinks<__half>(p, tq, tk, tv, to, block_size, grid, max_query_len, s);
}
}  // namespace pkv
