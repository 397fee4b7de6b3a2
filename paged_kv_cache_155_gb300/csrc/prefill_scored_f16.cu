// prefill_scored_f16.cu -- fp16 instantiations of the scored prefill kernels (capped and
// biased scores, interval masks).
#include "prefill_launch.cuh"

namespace pkv {
pkv_status launch_prefill_scored_f16(const PrefillParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                     const CUtensorMap &tv, const CUtensorMap &to, int block_size, int grid,
                                     int max_query_len, cudaStream_t s) {
    return launch_prefill<__half, true>(p, tq, tk, tv, to, block_size, grid, max_query_len, s);
}
}  // namespace pkv
