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

// Threads of a CTA: few tokens, whose CTAs all run at once, take kWide threads each (a
// token's rows in fewer steps); more take kNarrow, whose CTAs start and end in finer
// turns.  Measured, wide / narrow: 64 tokens of 32 + 2 x 8 heads of 128 3.1 us / 3.6, 800
// tokens 6.6 / 5.7, 8192 tokens 38 / 35; 8192 tokens into an INT8 cache 53 / 43.
constexpr int kWide = 256, kNarrow = 128;
// Steps of a thread whose loads are in flight together, and threads per SM (48 registers,
// 64 with the quantiser): the bytes in flight.  Measured on 8192 tokens of 64 + 2 x 8
// heads, wide CTAs: 59 us; four steps and 768 threads 68, one step and 1536 threads 70.
constexpr int kDepth = 2;
constexpr int kResident16 = 1280, kResidentInt8 = 1024;
// Tokens per CTA from kManyTokens tokens on: two share the angles' latency; below, one, so
// that the SMs share the work.  Chosen with wide CTAs (8192 tokens of 64 + 2 x 8 heads: 59.0 us,
// with one token 59.8, with four 61.9).  Narrow ones, which this range takes now, one token /
// two: the same 53.1 / 54.8, 4096 tokens 28.7 / 31.9; INT8 cache, 32 + 2 x 32 heads of 64, 8192
// tokens 52.2 / 50.2, 4096 25.6 / 24.7, 3000 19.9 / 21.5.
constexpr int kTok = 2, kManyTokens = 2048;

// quantize_int8 (pkv_device.cuh) without a division in most cases: the quotient by an
// approximate reciprocal is off by less than 2^-20 of itself, so its rounding to an
// integer is quantize_int8's unless it lies within 1e-3 of a tie (|quotient| <= 127:
// an error below 1.3e-4); those, and scales whose reciprocal could overflow or
// vanish, take the division.  Adding 1.5 * 2^23 rounds to nearest even and leaves the
// code in the low byte.
__device__ __forceinline__ uint32_t quantize_int8_byte(float x, float s) {
    const float q = fminf(fmaxf(x * pkv::fast_rcp(s), -127.f), 127.f);
    const float t = q + 12582912.f;
    const bool in_range = __float_as_uint(s) - 0x0d800000u < 0x64000000u;  // 2^-100 <= s < 2^100
    if (in_range && fabsf(q - (t - 12582912.f)) < 0.499f) return __float_as_uint(t) & 0xffu;
    return static_cast<uint32_t>(pkv::quantize_int8(x, s)) & 0xffu;
}

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
    int num_axes, pairs, num_q_heads, num_kv_heads;
    int block_shift;                                     // log2 of the block size
};

// Fraction of a turn that pair i of token n has made, as a signed 32-bit fixed-point
// fraction in [-1/2, 1/2).
__device__ __forceinline__ int turn_fraction(double inv_freq, int64_t position) {
    const double turns = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
    const double frac = turns - floor(turns);
    const uint64_t f = static_cast<uint64_t>(frac * 18446744073709551616.0);  // 2^64
    return static_cast<int>(static_cast<uint32_t>((static_cast<uint64_t>(position) * f) >> 32));
}

// One CTA per TOK consecutive tokens.  LANES = D / 16 threads share a row of one
// head, each taking two 16-byte vectors: pairs 8 c .. 8 c + 7 of the rotation (the
// vectors at channels 8 c and pairs + 8 c for split halves, 16 c and 16 c + 8 for
// adjacent channels) or two vectors behind the rotated channels, so that a thread's
// angles are the same in every row of a token and a rotation never crosses threads.
// The rows are the q heads, then K, then V; a thread's first rows are loaded before
// the angles are computed, one pair of one token per thread.
template <typename T, bool QUANT, int D, bool ADJACENT, int THREADS, int TOK>
__global__ void __launch_bounds__(THREADS, (QUANT ? kResidentInt8 : kResident16) / THREADS) rope_reshape_and_cache_kernel(const RopeParams p) {
    constexpr int LANES = D / 16;
    constexpr int ROWS = THREADS / LANES;  // rows in flight per step
    static_assert(TOK * (D / 2) <= THREADS, "one thread per angle");
    __shared__ float2 turn[TOK][D / 2];     // (cos, sin)
    __shared__ int64_t slots[TOK];          // -1: skip
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TOK;
    const int c = threadIdx.x % LANES;
    const int row0 = threadIdx.x / LANES;
    const int rows_q = p.num_q_heads, rows_k = rows_q + p.num_kv_heads, rows = rows_k + p.num_kv_heads;

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

    // The CTA's steps: step j is rows (j % steps) ROWS + row0 of token n0 + j / steps.
    // A thread keeps kDepth steps' loads in flight: those of step j + kDepth are issued
    // as step j's vectors have been used.
    const int steps = (rows + ROWS - 1) / ROWS;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TOK), p.num_tokens - n0));
    const char *q_row = p.q + n0 * p.q_stride, *k_row = p.k_new + n0 * p.k_stride, *v_row = p.v_new + n0 * p.v_stride;
    uint4 x0[kDepth], x1[kDepth];
    int lk = 0, lr = row0;  // token and row of the next load
    auto load = [&](int u) {
        if (lk < tokens && lr < rows) {  // (a skipped token's K and V rows are read for nothing)
            const char *src = lr < rows_q   ? q_row + lk * p.q_stride + lr * (2 * D)
                              : lr < rows_k ? k_row + lk * p.k_stride + (lr - rows_q) * (2 * D)
                                            : v_row + lk * p.v_stride + (lr - rows_k) * (2 * D);
            x0[u] = reinterpret_cast<const uint4 *>(src)[v0];
            x1[u] = reinterpret_cast<const uint4 *>(src)[v1];
        }
        lr += ROWS;
        if (lr >= steps * ROWS) {
            lr = row0;
            ++lk;
        }
    };
#pragma unroll
    for (int u = 0; u < kDepth; ++u) load(u);

    if (static_cast<int>(threadIdx.x) < tokens) {
        int64_t slot = p.slot_mapping[n0 + threadIdx.x];
        if (slot >= p.num_slots) {
            pkv::raise_flag(p.status, PKV_DEVERR_SLOT);
            slot = -1;
        }
        slots[threadIdx.x] = slot;
    }
    if (static_cast<int>(threadIdx.x) < TOK * (D / 2)) {
        const int i = threadIdx.x % (D / 2), k = threadIdx.x / (D / 2);
        if (i < p.pairs && k < tokens) {
            const int axis = p.axis_of_pair ? p.axis_of_pair[i] : 0;
            float2 cs = make_float2(1.f, 0.f);
            if (axis < 0 || axis >= p.num_axes) {
                if (n0 + k == 0) pkv::raise_flag(p.status, PKV_DEVERR_ROPE_AXIS);  // left unrotated
            } else {
                const int fr = turn_fraction(p.inv_freq[i], p.positions[axis * p.num_tokens + n0 + k]);
                sincospif(static_cast<float>(fr) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2 fr / 2^32
            }
            turn[k][(i % 8) * LANES + i / 8] = cs;  // a row's lanes read consecutive words
        }
    }
    __syncthreads();

    auto process = [&](uint4 y0, uint4 y1, int k, int r) {
        const int64_t slot = slots[k];
        if (r >= rows || (slot < 0 && r >= rows_q)) return;  // a skipped token still gets its rotated q
        float f0[8], f1[8];
        const bool turned = rotates && r < rows_k;
        if (turned || (QUANT && r >= rows_q)) {
            pkv::Elem<T>::to_f32x8(y0, f0);
            pkv::Elem<T>::to_f32x8(y1, f1);
        }
        if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = turn[k][e * LANES + c];
                // split halves: pair e is (f0[e], f1[e]); adjacent: channels 2 e, 2 e + 1 of the 16
                float &a = ADJACENT ? (e < 4 ? f0[(2 * e) & 7] : f1[(2 * e) & 7]) : f0[e];
                float &b = ADJACENT ? (e < 4 ? f0[(2 * e + 1) & 7] : f1[(2 * e + 1) & 7]) : f1[e];
                const float a0 = a, b0 = b;
                a = a0 * cs.x - b0 * cs.y;
                b = b0 * cs.x + a0 * cs.y;
            }
            if (!QUANT || r < rows_q) {
                y0 = make_uint4(pkv::Elem<T>::pack2(f0[0], f0[1]), pkv::Elem<T>::pack2(f0[2], f0[3]),
                                pkv::Elem<T>::pack2(f0[4], f0[5]), pkv::Elem<T>::pack2(f0[6], f0[7]));
                y1 = make_uint4(pkv::Elem<T>::pack2(f1[0], f1[1]), pkv::Elem<T>::pack2(f1[2], f1[3]),
                                pkv::Elem<T>::pack2(f1[4], f1[5]), pkv::Elem<T>::pack2(f1[6], f1[7]));
            }
        }
        if (r < rows_q) {
            uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + (n0 + k) * p.q_out_stride + r * (2 * D));
            dst[v0] = y0;
            dst[v1] = y1;
            return;
        }
        const bool is_v = r >= rows_k;
        const int h = is_v ? r - rows_k : r - rows_q;
        const int64_t blk = slot >> p.block_shift;
        const int off = static_cast<int>(slot & ((1 << p.block_shift) - 1));
        char *row = (is_v ? p.v_cache : p.k_cache) + blk * p.block_stride +
                    ((static_cast<int64_t>(h) << p.block_shift) + off) * (D * (QUANT ? 1 : 2));
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
                    w[e / 4] |= quantize_int8_byte(f[e], s[e]) << (8 * (e % 4));
                reinterpret_cast<uint2 *>(row)[v] = make_uint2(w[0], w[1]);
            }
        } else {
            reinterpret_cast<uint4 *>(row)[v0] = y0;
            reinterpret_cast<uint4 *>(row)[v1] = y1;
        }
    };
    int k = 0, r = row0;
    while (k < tokens) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (k < tokens) process(x0[u], x1[u], k, r);
            load(u);
            r += ROWS;
            if (r >= steps * ROWS) {
                r = row0;
                ++k;
            }
        }
    }
}

template <typename T, bool QUANT, int D, bool ADJACENT>
void launch_rope_form(const RopeParams &p, int sms, cudaStream_t s) {
    const unsigned tokens = static_cast<unsigned>(p.num_tokens);
    if (p.num_tokens <= static_cast<int64_t>(sms) * (QUANT ? kResidentInt8 : kResident16) / kWide)
        rope_reshape_and_cache_kernel<T, QUANT, D, ADJACENT, kWide, 1><<<tokens, kWide, 0, s>>>(p);
    else if (p.num_tokens < kManyTokens)
        rope_reshape_and_cache_kernel<T, QUANT, D, ADJACENT, kNarrow, 1><<<tokens, kNarrow, 0, s>>>(p);
    else
        rope_reshape_and_cache_kernel<T, QUANT, D, ADJACENT, kNarrow, kTok><<<(tokens + kTok - 1) / kTok, kNarrow, 0, s>>>(p);
}

template <typename T, bool QUANT>
void launch_rope(const RopeParams &p, int head_dim, bool adjacent, int sms, cudaStream_t s) {
    if (head_dim == 128) {
        if (adjacent) launch_rope_form<T, QUANT, 128, true>(p, sms, s);
        else launch_rope_form<T, QUANT, 128, false>(p, sms, s);
    } else {
        if (adjacent) launch_rope_form<T, QUANT, 64, true>(p, sms, s);
        else launch_rope_form<T, QUANT, 64, false>(p, sms, s);
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
    const int sms = pkv::current_sm_count();
    if (!status || sms <= 0) return PKV_ERR_CUDA;
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
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool adjacent = interleaved != 0;
    if (dtype == PKV_F16) {
        if (int8_kv) launch_rope<__half, true>(p, head_dim, adjacent, sms, s);
        else launch_rope<__half, false>(p, head_dim, adjacent, sms, s);
    } else {
        if (int8_kv) launch_rope<__nv_bfloat16, true>(p, head_dim, adjacent, sms, s);
        else launch_rope<__nv_bfloat16, false>(p, head_dim, adjacent, sms, s);
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
