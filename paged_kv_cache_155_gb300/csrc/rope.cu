// rope.cu -- rotary positions with one to four axes, fused with the cache write:
//   pkv_rope_reshape_and_cache       16-bit cache
//   pkv_rope_reshape_and_cache_int8  INT8 cache with per-channel scales
//
// For token n, pair i of the rotated channels turns by
//     angle = positions[axis_of_pair[i]][n] * inv_freq[i],
//     (a, b) -> (a cos - b sin, b cos + a sin),
// in q (written to q_out) and in the new K row, which goes to its cache slot with
// the V row beside it.  Images and video give a token several positions (time,
// height, width); each pair follows one of them.
//
// The angle is reduced to a fraction of a turn in 64-bit integers: with
// f = floor(2^64 frac(inv_freq / 2 pi)), the product positions * f modulo 2^64 is
// the fraction of the turn (whole turns fall off the top), so a far position loses
// nothing: the error is |position| * 2^-53 turns, that of inv_freq / 2 pi in 64
// bits.  A float product loses the angle itself at 2^24 / 2 pi turns.  The
// fraction's top 32 bits, rounded to fp32, then go through sincospif (sine and cosine
// off by less than 2^-21).
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // rows of a thread whose loads are in flight together
constexpr int kMaxPairs = 64;   // head_dim / 2

struct RopeParams {
    const char *q, *k_new, *v_new;  // rows of [heads][head_dim]
    char *q_out, *k_cache, *v_cache;
    const int64_t *positions;       // [num_axes][num_tokens]
    const int32_t *axis_of_pair;    // [pairs] or null (axis 0)
    const double *inv_freq;         // [pairs]
    const int64_t *slot_mapping;
    const float *k_scale, *v_scale; // INT8 cache
    unsigned int *status;
    int64_t num_tokens;
    int64_t q_stride, k_stride, v_stride, q_out_stride;  // bytes between tokens
    int64_t num_slots, block_stride;                     // block_stride in bytes
    int num_axes, pairs, num_q_heads, num_kv_heads, block_size;
};

// Fraction of a turn that pair i of token n has made, as a signed 32-bit fixed-point
// fraction in [-1/2, 1/2).
__device__ __forceinline__ int turn_fraction(double inv_freq, int64_t position) {
    const double turns = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
    const double frac = turns - floor(turns);
    const uint64_t f = static_cast<uint64_t>(frac * 18446744073709551616.0);  // 2^64
    return static_cast<int>(static_cast<uint32_t>((static_cast<uint64_t>(position) * f) >> 32));
}

// One CTA per token.  LANES = D / 16 threads share a row of one head, each taking
// two 16-byte vectors: pairs 8 c .. 8 c + 7 of the rotation (the vectors at channels
// 8 c and pairs + 8 c for split halves, 16 c and 16 c + 8 for adjacent channels) or
// two vectors behind the rotated channels, so that a thread's angles are the same
// in every row and a rotation never crosses threads.  The rows are the q heads,
// then K, then V; the loads of a thread's first rows are issued before the angles
// are computed.
template <typename T, bool QUANT, int D, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) rope_reshape_and_cache_kernel(const RopeParams p) {
    constexpr int LANES = D / 16;
    constexpr int ROWS = kThreads / LANES;  // rows in flight per step
    __shared__ float2 turn[kMaxPairs];      // (cos, sin)
    const int64_t n = blockIdx.x;
    const int c = threadIdx.x % LANES;
    const int row0 = threadIdx.x / LANES;
    const int rows_q = p.num_q_heads, rows_k = rows_q + p.num_kv_heads, rows = rows_k + p.num_kv_heads;

    const int64_t slot = p.slot_mapping[n];
    const bool store_kv = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0) pkv::raise_flag(p.status, PKV_DEVERR_SLOT);
    const int last = store_kv ? rows : rows_q;  // a skipped token still gets its rotated q

    // this thread's two vectors of a row, in 16-byte units
    const int groups = p.pairs / 8;  // rotation groups of 8 pairs
    const bool rotates = c < groups;
    int v0, v1;
    if (ADJACENT) {
        v0 = 2 * c;
        v1 = 2 * c + 1;
    } else {
        v0 = rotates ? c : 2 * c;        // behind the rotation: 2 groups + 2 (c - groups)
        v1 = rotates ? c + groups : 2 * c + 1;
    }

    auto source = [&](int r) -> const uint4 * {
        if (r < rows_q) return reinterpret_cast<const uint4 *>(p.q + n * p.q_stride) + r * (D / 8);
        if (r < rows_k) return reinterpret_cast<const uint4 *>(p.k_new + n * p.k_stride) + (r - rows_q) * (D / 8);
        return reinterpret_cast<const uint4 *>(p.v_new + n * p.v_stride) + (r - rows_k) * (D / 8);
    };
    uint4 x0[kUnroll], x1[kUnroll];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = base + u * ROWS;
            if (r < last) {
                const uint4 *src = source(r);
                x0[u] = src[v0];
                x1[u] = src[v1];
            }
        }
    };
    load(row0);

    if (static_cast<int>(threadIdx.x) < p.pairs) {
        int axis = p.axis_of_pair ? p.axis_of_pair[threadIdx.x] : 0;
        float2 cs = make_float2(1.f, 0.f);
        if (axis < 0 || axis >= p.num_axes) {
            if (n == 0) pkv::raise_flag(p.status, PKV_DEVERR_ROPE_AXIS);  // left unrotated
        } else {
            const int fr = turn_fraction(p.inv_freq[threadIdx.x], p.positions[axis * p.num_tokens + n]);
            sincospif(static_cast<float>(fr) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2 fr / 2^32
        }
        turn[threadIdx.x] = cs;
    }
    __syncthreads();
    float cosv[8], sinv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 cs = rotates ? turn[8 * c + e] : make_float2(1.f, 0.f);
        cosv[e] = cs.x;
        sinv[e] = cs.y;
    }

    const int64_t blk = store_kv ? slot / p.block_size : 0;
    const int off = store_kv ? static_cast<int>(slot - blk * p.block_size) : 0;
    for (int base = row0; base < last; base += kUnroll * ROWS) {
        if (base != row0) load(base);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = base + u * ROWS;
            if (r >= last) break;
            uint4 y0 = x0[u], y1 = x1[u];
            float f0[8], f1[8];
            const bool turned = rotates && r < rows_k;
            if (turned || (QUANT && r >= rows_q)) {
                pkv::Elem<T>::to_f32x8(y0, f0);
                pkv::Elem<T>::to_f32x8(y1, f1);
            }
            if (turned) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // split halves: pair e is (f0[e], f1[e]); adjacent: channels 2 e, 2 e + 1 of the 16
                    float &a = ADJACENT ? (e < 4 ? f0[(2 * e) & 7] : f1[(2 * e) & 7]) : f0[e];
                    float &b = ADJACENT ? (e < 4 ? f0[(2 * e + 1) & 7] : f1[(2 * e + 1) & 7]) : f1[e];
                    const float a0 = a, b0 = b;
                    a = a0 * cosv[e] - b0 * sinv[e];
                    b = b0 * cosv[e] + a0 * sinv[e];
                }
                if (!QUANT || r < rows_q) {
                    y0 = make_uint4(pkv::Elem<T>::pack2(f0[0], f0[1]), pkv::Elem<T>::pack2(f0[2], f0[3]),
                                    pkv::Elem<T>::pack2(f0[4], f0[5]), pkv::Elem<T>::pack2(f0[6], f0[7]));
                    y1 = make_uint4(pkv::Elem<T>::pack2(f1[0], f1[1]), pkv::Elem<T>::pack2(f1[2], f1[3]),
                                    pkv::Elem<T>::pack2(f1[4], f1[5]), pkv::Elem<T>::pack2(f1[6], f1[7]));
                }
            }
            if (r < rows_q) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + n * p.q_out_stride) + r * (D / 8);
                dst[v0] = y0;
                dst[v1] = y1;
                continue;
            }
            const bool is_v = r >= rows_k;
            const int h = is_v ? r - rows_k : r - rows_q;
            char *row = (is_v ? p.v_cache : p.k_cache) + blk * p.block_stride +
                        (static_cast<int64_t>(h) * p.block_size + off) * (D * (QUANT ? 1 : 2));
            if constexpr (QUANT) {
                const float *scale = (is_v ? p.v_scale : p.k_scale) + h * D;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int v = half ? v1 : v0;
                    const float *f = half ? f1 : f0;
                    const float4 sa = reinterpret_cast<const float4 *>(scale)[2 * v];
                    const float4 sb = reinterpret_cast<const float4 *>(scale)[2 * v + 1];
                    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
                    uint32_t w[2] = {0u, 0u};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e / 4] |= (static_cast<uint32_t>(pkv::quantize_int8(f[e], s[e])) & 0xffu) << (8 * (e % 4));
                    reinterpret_cast<uint2 *>(row)[v] = make_uint2(w[0], w[1]);
                }
            } else {
                reinterpret_cast<uint4 *>(row)[v0] = y0;
                reinterpret_cast<uint4 *>(row)[v1] = y1;
            }
        }
    }
}

template <typename T, bool QUANT>
void launch_rope(const RopeParams &p, int head_dim, bool adjacent, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.num_tokens);
    if (head_dim == 128) {
        if (adjacent) rope_reshape_and_cache_kernel<T, QUANT, 128, true><<<grid, kThreads, 0, s>>>(p);
        else rope_reshape_and_cache_kernel<T, QUANT, 128, false><<<grid, kThreads, 0, s>>>(p);
    } else {
        if (adjacent) rope_reshape_and_cache_kernel<T, QUANT, 64, true><<<grid, kThreads, 0, s>>>(p);
        else rope_reshape_and_cache_kernel<T, QUANT, 64, false><<<grid, kThreads, 0, s>>>(p);
    }
}

pkv_status rope_impl(const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
                     int64_t v_stride, const int64_t *positions, int num_axes, const int32_t *axis_of_pair,
                     const double *inv_freq, int rotary_dim, int interleaved, const int64_t *slot_mapping,
                     int64_t num_tokens, void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
                     int64_t num_blocks, int64_t block_stride_elems, int num_q_heads, int num_kv_heads,
                     int head_dim, int block_size, bool int8_kv, const float *k_scale, const float *v_scale,
                     pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim % 16) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > head_dim || num_axes < 1 || num_axes > 4 || num_tokens < 0 ||
        num_tokens > 0x7fffffffLL || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
        num_q_heads > 65535 || num_kv_heads > 65535)
        return PKV_ERR_INVALID_ARG;
    const int64_t half_elems = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_elems < half_elems || block_stride_elems % (int8_kv ? 16 : 8)) return PKV_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (q_stride < q_row || q_out_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 ||
        q_out_stride % 8 || k_stride % 8 || v_stride % 8)
        return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (int8_kv && (!k_scale || !v_scale || !pkv::aligned16(k_scale) || !pkv::aligned16(v_scale)))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k_new || !v_new || !q_out || !positions || !inv_freq || !slot_mapping || !pkv::aligned16(q) ||
        !pkv::aligned16(k_new) || !pkv::aligned16(v_new) || !pkv::aligned16(q_out) ||
        ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq) |
          reinterpret_cast<uintptr_t>(slot_mapping)) & 7u) ||
        (reinterpret_cast<uintptr_t>(axis_of_pair) & 3u))
        return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    RopeParams p{};
    p.q = static_cast<const char *>(q);
    p.k_new = static_cast<const char *>(k_new);
    p.v_new = static_cast<const char *>(v_new);
    p.q_out = static_cast<char *>(q_out);
    p.k_cache = static_cast<char *>(k_cache);
    p.v_cache = static_cast<char *>(v_cache);
    p.positions = positions;
    p.axis_of_pair = axis_of_pair;
    p.inv_freq = inv_freq;
    p.slot_mapping = slot_mapping;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.status = status;
    p.num_tokens = num_tokens;
    p.q_stride = q_stride * 2;
    p.k_stride = k_stride * 2;
    p.v_stride = v_stride * 2;
    p.q_out_stride = q_out_stride * 2;
    p.num_slots = num_blocks * block_size;
    p.block_stride = block_stride_elems * (int8_kv ? 1 : 2);
    p.num_axes = num_axes;
    p.pairs = rotary_dim / 2;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool adjacent = interleaved != 0;
    if (dtype == PKV_F16) {
        if (int8_kv) launch_rope<__half, true>(p, head_dim, adjacent, s);
        else launch_rope<__half, false>(p, head_dim, adjacent, s);
    } else {
        if (int8_kv) launch_rope<__nv_bfloat16, true>(p, head_dim, adjacent, s);
        else launch_rope<__nv_bfloat16, false>(p, head_dim, adjacent, s);
    }
    pkv::count_launch();
    return pkv::launch_status();
}

}  // namespace

extern "C" {

PKV_API pkv_status pkv_rope_reshape_and_cache(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
    const int64_t *positions, int num_axes, const int32_t *axis_of_pair, const double *inv_freq, int rotary_dim,
    int interleaved, const int64_t *slot_mapping, int64_t num_tokens, void *q_out, int64_t q_out_stride,
    void *k_cache, void *v_cache, int64_t num_blocks, int64_t block_stride_elems, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, pkv_dtype dtype, void *stream) {
    return rope_impl(q, q_stride, k_new, k_stride, v_new, v_stride, positions, num_axes, axis_of_pair, inv_freq,
                     rotary_dim, interleaved, slot_mapping, num_tokens, q_out, q_out_stride, k_cache, v_cache,
                     num_blocks, block_stride_elems, num_q_heads, num_kv_heads, head_dim, block_size, false,
                     nullptr, nullptr, dtype, stream);
}

PKV_API pkv_status pkv_rope_reshape_and_cache_int8(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
    const int64_t *positions, int num_axes, const int32_t *axis_of_pair, const double *inv_freq, int rotary_dim,
    int interleaved, const int64_t *slot_mapping, int64_t num_tokens, void *q_out, int64_t q_out_stride,
    int8_t *k_cache, int8_t *v_cache, int64_t num_blocks, int64_t block_stride_elems, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, const float *k_scale, const float *v_scale, pkv_dtype dtype,
    void *stream) {
    return rope_impl(q, q_stride, k_new, k_stride, v_new, v_stride, positions, num_axes, axis_of_pair, inv_freq,
                     rotary_dim, interleaved, slot_mapping, num_tokens, q_out, q_out_stride, k_cache, v_cache,
                     num_blocks, block_stride_elems, num_q_heads, num_kv_heads, head_dim, block_size, true,
                     k_scale, v_scale, dtype, stream);
}

}  // extern "C"
