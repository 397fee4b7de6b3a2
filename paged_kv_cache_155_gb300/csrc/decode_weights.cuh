// decode_weights.cuh -- what follows the scored decode: the merge of its partitions and
// the accumulated attention weights, in one launch.
#pragma once

#include "decode_kernel.cuh"

namespace pkv {

// weights_out[b][h][t] = weights[b][h][t] + the sum over KV head h's query heads of their
// softmax weights 2^(s - M) / L at token t, for every t of the context (masked tokens
// keep their weight).  The decode kernel left the scores s, each partition's maximum and its
// sum of unrounded exponentials.
struct WeightParams {
    const float *weights;  // or null: zeros
    float *weights_out;    // null: the merge alone
    int64_t weights_stride;
    int steps;             // kWeightStep-token steps per block, up to kMaxWeightSteps
    int chunks;            // blocks per (sequence, KV head), of steps steps each
    int vectors;           // rows of weights start 16-byte aligned
};
constexpr int kWeightThreads = 128;
constexpr int kWeightStep = 4 * kWeightThreads;   // four tokens per thread
// Steps of a block: they share the joining of the partitions, but a small batch needs its
// blocks on every SM (two contexts of 32768 tokens and 8 KV heads, 1024 steps: 64 us for
// the decode and its weights with four steps a block, 61 with one).
constexpr int kMaxWeightSteps = 4;
constexpr int kWeightBlocksPerSm = 8;
constexpr int kMaxWeightHeads = 128;  // query heads per KV head

// Maximum and sum of one row over its partitions, by a warp: every lane gets M and L.
__device__ __forceinline__ void join_row(const DecodeParams &p, int64_t row, int nparts, float &m, float &l) {
    const int lane = threadIdx.x & 31;
    const int64_t base = row * p.num_partitions;
    const float *sums = weight_sums(p, row);
    float mq = -INFINITY, lq = 0.f;
    if (lane < nparts) {
        mq = p.ws_m[base + lane];
        lq = sums[lane];
    }
    m = mq;
    for (int q = lane + 32; q < nparts; q += 32) m = fmaxf(m, p.ws_m[base + q]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    l = mq == -INFINITY ? 0.f : fast_exp2(mq - m) * lq;
    for (int q = lane + 32; q < nparts; q += 32) {
        const float mo = p.ws_m[base + q];
        if (mo != -INFINITY) l += fast_exp2(mo - m) * sums[q];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
}

// The weights of one chunk: four consecutive tokens per thread and step, the scores of
// four heads in flight; the first four are on their way while the block joins its heads'
// partitions.  What the decode kernel does not write -- lengths and old weights -- is
// read before the wait for it.
__device__ __forceinline__ void weights_chunk(const DecodeParams &p, const WeightParams &w, int idx) {
    __shared__ float head_max[kMaxWeightHeads], head_inv[kMaxWeightHeads];
    const int num_kv_heads = p.num_q_heads / p.group;
    const int t0 = idx % w.chunks * (w.steps * kWeightStep);
    const int kvh = idx / w.chunks % num_kv_heads, seq = idx / w.chunks / num_kv_heads;
    const int warp = threadIdx.x >> 5;
    int len = p.context_lens[seq];
    if (len < 0) len = 0;
    if (len > p.len_cap) len = p.len_cap;
    if (t0 >= len) return;  // uniform over the block
    const DecodeSpan span = span_of(p, seq, len);
    const int nparts = partitions_of_span(p, span, len);
    const int64_t row0 = static_cast<int64_t>(seq) * p.num_q_heads + kvh * p.group;
    const int64_t out_row = (static_cast<int64_t>(seq) * num_kv_heads + kvh) * w.weights_stride;
    const int t1 = min(len, t0 + w.steps * kWeightStep);
    const int first = t0 + 4 * static_cast<int>(threadIdx.x);
    float4 old[kMaxWeightSteps];
#pragma unroll
    for (int i = 0; i < kMaxWeightSteps; ++i) {
        const int t = first + i * kWeightStep;
        old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!w.weights || t >= t1) continue;
        const float *src = w.weights + out_row + t;
        if (w.vectors && t + 4 <= len) {
            old[i] = *reinterpret_cast<const float4 *>(src);
        } else {
            old[i].x = src[0];
            if (t + 1 < len) old[i].y = src[1];
            if (t + 2 < len) old[i].z = src[2];
            if (t + 3 < len) old[i].w = src[3];
        }
    }
    pdl_wait();
    // a span that is not empty begins at a multiple of 8 and the rows of scores at multiples
    // of 32, so four tokens are one aligned vector; it may start before the first visible
    // token (-inf) or reach past the context
    const auto inside = [&](int t) { return t < t1 && t + 4 > span.lo && span.begin < len; };
    const float *scores = p.ws_s + row0 * p.score_stride - span.begin;
    float4 s[4];
    const auto load = [&](int t, int g0) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (inside(t) && g0 + g < p.group) s[g] = *reinterpret_cast<const float4 *>(scores + (g0 + g) * p.score_stride + t);
    };
    load(first, 0);
    for (int g = warp; g < p.group; g += kWeightThreads / 32) {
        float m, l;
        join_row(p, row0 + g, nparts, m, l);
        if ((threadIdx.x & 31) == 0) {
            head_max[g] = m == -INFINITY ? 0.f : m;  // an empty row: every score is -inf, every weight 0
            head_inv[g] = l > 0.f ? 1.f / l : 0.f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxWeightSteps; ++i) {
        const int t = first + i * kWeightStep;
        if (t >= t1) return;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (inside(t)) {
            for (int g0 = 0; g0 < p.group; g0 += 4) {
                if (g0 > 0) load(t, g0);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g0 + g >= p.group) break;
                    const float m = head_max[g0 + g], inv = head_inv[g0 + g];
                    sum.x = fmaf(fast_exp2(s[g].x - m), inv, sum.x);
                    sum.y = fmaf(fast_exp2(s[g].y - m), inv, sum.y);
                    sum.z = fmaf(fast_exp2(s[g].z - m), inv, sum.z);
                    sum.w = fmaf(fast_exp2(s[g].w - m), inv, sum.w);
                }
            }
        }
        load(t + kWeightStep, 0);
        sum = make_float4(old[i].x + sum.x, old[i].y + sum.y, old[i].z + sum.z, old[i].w + sum.w);
        float *dst = w.weights_out + out_row + t;
        if (w.vectors && t + 4 <= len) {
            *reinterpret_cast<float4 *>(dst) = sum;
        } else {
            dst[0] = sum.x;
            if (t + 1 < len) dst[1] = sum.y;
            if (t + 2 < len) dst[2] = sum.z;
            if (t + 3 < len) dst[3] = sum.w;
        }
    }
}

// The first merge_blocks blocks merge the partitions (paged_decode_merge_kernel's work),
// the others take a chunk of weights each.  Launched behind the decode kernel as its
// programmatic dependent.  Bound by latency and the scores' 4 bytes per query head and
// token, written by the decode and read back (mostly from L2): 64 ragged contexts of 32 / 8
// heads take 168 us without and 190 us with their weights.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(kWeightThreads) paged_decode_scored_tail_kernel(const DecodeParams p, int num_rows,
                                                                                  int merge_blocks, const WeightParams w) {
    if (static_cast<int>(blockIdx.x) < merge_blocks) {
        pdl_wait();
        merge_rows<T, D, WPR, true>(p, num_rows, blockIdx.x);
    } else {
        weights_chunk(p, w, static_cast<int>(blockIdx.x) - merge_blocks);
    }
}

}  // namespace pkv
