// decode_weights.cuh -- the accumulated attention weights of the scored decode.
#pragma once

#include "decode_kernel.cuh"

namespace pkv {

// The scored decode's accumulated weights: weights_out[b][h][t] = weights[b][h][t] +
// the sum over KV head h's query heads of their softmax weights 2^(s - M) / L at token
// t, for every t of the context (masked tokens keep their weight).  The decode kernel
// left the scores s and each partition's (m, l); a block first joins the partitions of
// its heads to M and 1 / L, as the merge does, then takes kWeightTokens tokens.
// Bound by the scores' bytes (4 per query head and token, mostly still in L2) and the
// two fp32 arrays.  Launched behind the decode as its programmatic dependent.
struct WeightParams {
    const float *weights;  // or null: zeros
    float *weights_out;
    int64_t weights_stride;
};
constexpr int kWeightThreads = 128;
constexpr int kWeightTokens = 4 * kWeightThreads;
constexpr int kMaxWeightHeads = 128;  // query heads per KV head

__global__ void __launch_bounds__(kWeightThreads) decode_weights_kernel(const DecodeParams p, const WeightParams w) {
    __shared__ float head_max[kMaxWeightHeads], head_inv[kMaxWeightHeads];
    const int seq = blockIdx.z, kvh = blockIdx.y, t0 = blockIdx.x * kWeightTokens;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int len = p.context_lens[seq];
    if (len < 0) len = 0;
    if (len > p.len_cap) len = p.len_cap;
    if (t0 >= len) return;  // uniform over the block
    const DecodeSpan span = span_of(p, seq, len);
    const int nparts = partitions_of_span(p, span, len);
    const int64_t row0 = static_cast<int64_t>(seq) * p.num_q_heads + kvh * p.group;
    for (int g = warp; g < p.group; g += kWeightThreads / 32) {
        const int64_t base = (row0 + g) * p.num_partitions;
        float m = -INFINITY, l = 0.f;
        for (int q = lane; q < nparts; q += 32) m = fmaxf(m, p.ws_m[base + q]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int q = lane; q < nparts; q += 32) {
            const float mq = p.ws_m[base + q];
            if (mq != -INFINITY) l += fast_exp2(mq - m) * p.ws_l[base + q];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            head_max[g] = m == -INFINITY ? 0.f : m;  // an empty row: every score is -inf, every weight 0
            head_inv[g] = l > 0.f ? 1.f / l : 0.f;
        }
    }
    __syncthreads();
    const int64_t wrow = (static_cast<int64_t>(seq) * (p.num_q_heads / p.group) + kvh) * w.weights_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + i * kWeightThreads + threadIdx.x;
        if (t >= len) break;
        float sum = 0.f;
        if (t >= span.lo) {
            const float *s = p.ws_s + row0 * p.score_stride + (t - span.begin);
            for (int g = 0; g < p.group; ++g) sum = fmaf(fast_exp2(s[g * p.score_stride] - head_max[g]), head_inv[g], sum);
        }
        w.weights_out[wrow + t] = w.weights ? w.weights[wrow + t] + sum : sum;
    }
}

}  // namespace pkv
