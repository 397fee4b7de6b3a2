// int4_cache.cu -- the 4-bit cache's write and read-back (format: int4.cuh):
//   pkv_reshape_and_cache_int4    quantise each new token's K/V rows into its slot
//   pkv_dequantise_blocks_int4    blocks of a 4-bit pool -> blocks of a 16-bit pool
// Both move a few bytes per value and are bound by memory: 2 + 5/8 bytes a value each way.
#include <type_traits>

#include "int4.cuh"
#include "pkv_host.h"

namespace {

// The nearest code of a value d above its group's zero, as a float, ties to the even code: the
// quotient by an approximate reciprocal is off by less than one code, and the remainder d - r s,
// exact in one FMA, says whether the next code is nearer.  (16-bit values often lie exactly halfway,
// so the remainder decides, not the rounded quotient.)  A remainder of half a step moves an odd code
// only: even codes compare with the next float above it.  Adding 1.5 * 2^23 rounds to nearest and
// shows the code's last bit.  A NaN gets 0.
__device__ __forceinline__ float int4_code(float d, float s, float rcp, float half_odd, float half_even) {
    d = fmaxf(d, 0.f);
    const float t = fmaf(d, rcp, 12582912.f);
    const float r = t - 12582912.f;
    const float e = fmaf(-r, s, d);
    const float half = __float_as_uint(t) & 1u ? half_odd : half_even;
    return fabsf(e) >= half ? r + copysignf(1.f, e) : r;
}

// Four codes as floats -> one 16-bit word, the first in its low nibble.
__device__ __forceinline__ uint32_t int4_word(const float *c) {
    const float v = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]);  // < 2^16, exact
    return __float_as_uint(v + 8388608.f) & 0xffffu;
}

// (smallest, largest) of a group's 32 values, 8 in each of four lanes, packed in the rows' type; NaNs lose.
template <typename T>
__device__ __forceinline__ void int4_range(const uint4 &row, float &lo, float &hi) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 *v = reinterpret_cast<const T2 *>(&row);
    const T2 least = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
    const T2 most = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    // the smallest value in the low half, the largest one's negative in the high half
    T2 m;
    m.x = __hmin(least.x, least.y);
    m.y = __hneg(__hmax(most.x, most.y));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&m), o);
        m = __hmin2(m, *reinterpret_cast<const T2 *>(&other));
    }
    const float2 f = pkv::Int4Param<T>::unpack(*reinterpret_cast<const uint32_t *>(&m));
    lo = f.x;
    hi = -f.y;
}

// Quantises the 8 channels 8 i .. 8 i + 7 of a group whose four lanes call together: the
// two 16-bit code words of its units 2 i and 2 i + 1, and the group's (s, z) word.
template <typename T>
__device__ __forceinline__ void int4_quantise(const uint4 &row, uint32_t &unit0, uint32_t &unit1, uint32_t &param) {
    float f[8], lo, hi;
    pkv::Elem<T>::to_f32x8(row, f);
    int4_range<T>(row, lo, hi);
    // the smallest scale with 15 s >= hi - lo: a number of the type that is surely not above it, then
    // up while 15 s (exact) is too small
    const float range = __fsub_ru(hi, lo);
    uint32_t sb = pkv::Int4Param<T>::scale_down(range * 0.06666663f);
    if (15.f * pkv::Int4Param<T>::value(sb) < range) ++sb;
    if (15.f * pkv::Int4Param<T>::value(sb) < range) ++sb;
    const float s = pkv::Int4Param<T>::value(sb);
    param = sb | (pkv::Int4Param<T>::bits(lo) << 16);
    // scales whose reciprocal would overflow or vanish (zero among them) take the division
    const bool in_range = __float_as_uint(s) - 0x0d800000u < 0x64000000u;  // 2^-100 <= s < 2^100
    float c[8];
    if (__all_sync(0xffffffffu, in_range)) {
        const float rcp = pkv::fast_rcp(s), half = 0.5f * s, above = half * 1.00000012f;
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = int4_code(f[e] - lo, s, rcp, half, above);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = fminf(fmaxf(rintf(__fdiv_rn(f[e] - lo, s)), 0.f), 15.f);
    }
    unit0 = int4_word(c);
    unit1 = int4_word(c + 4);
}

// A thread quantises 8 channels of one row of K and of V; the rows of a token and then the
// tokens follow one another.  Lanes 4 j + i hold channels 8 i .. of group j; lanes of groups j and
// j ^ 1 trade a word, so that each stores one 32-bit word of codes (a row's are contiguous).  Bound by
// arithmetic, some 13 operations a value: 8192 tokens of 8 heads of 128, bf16 15.3 us (with packed
// minima, one FMA per rounding and codes packed by FMAs; with a division, conversions and a CTA per token 22 us).
constexpr int kWriteThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads) reshape_and_cache_int4_kernel(
    const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, const int64_t *__restrict__ slot_mapping,
    char *__restrict__ k_cache, char *__restrict__ v_cache, int64_t num_slots, int64_t block_stride, int num_rows,
    int num_kv_heads, int block_shift, unsigned int *status) {
    constexpr int LANES = D / 8, NG = D / 32;
    const int row = blockIdx.x * (kWriteThreads / LANES) + threadIdx.x / LANES;  // token * num_kv_heads + head
    const int lane = threadIdx.x % LANES, j = lane / 4, u = 2 * (lane % 4);
    const bool there = row < num_rows;
    uint4 x[2] = {};
    int64_t slot = -1;
    const int n = row / num_kv_heads, h = row - n * num_kv_heads;
    if (there) {
        x[0] = k_new[static_cast<int64_t>(row) * LANES + lane];
        x[1] = v_new[static_cast<int64_t>(row) * LANES + lane];
        slot = slot_mapping[n];
    }
    if (slot >= num_slots) {
        if (h == 0 && lane == 0) pkv::raise_flag(status, PKV_DEVERR_SLOT);
        slot = -1;
    }
    const int bs = 1 << block_shift, off = static_cast<int>(slot) & (bs - 1);
    const int64_t at = (slot >> block_shift) * block_stride + static_cast<int64_t>(h) * pkv::int4_record_bytes(D, bs);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t unit0, unit1, param;
        int4_quantise<T>(x[half], unit0, unit1, param);
        const bool odd = j & 1;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? unit0 : unit1, 4);
        const uint32_t word = odd ? (other | (unit1 << 16)) : (unit0 | (other << 16));
        if (slot >= 0) {
            char *base = (half ? v_cache : k_cache) + at;
            *reinterpret_cast<uint32_t *>(base + off * (D / 2) + ((u + odd) * NG + (j & ~1)) * 2) = word;
            if (u == 0) *reinterpret_cast<uint32_t *>(base + bs * (D / 2) + off * (D / 8) + j * 4) = param;
        }
    }
}

constexpr int kReadThreads = 256;
constexpr int kReadDepth = 4;  // vectors of a thread in flight

// grid.x = pair, grid.y = chunk of a half block's vectors, grid.z = K (0) / V (1); a
// thread writes 8 channels (16 bytes) of a row, lanes as in the write.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) dequantise_blocks_int4_kernel(
    const char *__restrict__ k4, const char *__restrict__ v4, int64_t num_blocks4, int64_t block_stride4,
    const int64_t *__restrict__ pairs, uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache, int64_t num_blocks,
    int64_t block_stride_vecs, int num_kv_heads, int block_shift, unsigned int *status) {
    constexpr int LANES = D / 8, NG = D / 32;
    const int64_t src = pairs[2 * static_cast<int64_t>(blockIdx.x)], dst = pairs[2 * static_cast<int64_t>(blockIdx.x) + 1];
    if (src < 0 || src >= num_blocks4 || dst < 0 || dst >= num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) pkv::raise_flag(status, PKV_DEVERR_COPY_PAIR);
        return;
    }
    const int bs = 1 << block_shift;
    const int record = pkv::int4_record_bytes(D, bs);
    const char *from = (blockIdx.z ? v4 : k4) + src * block_stride4;
    uint4 *to = (blockIdx.z ? v_cache : k_cache) + dst * block_stride_vecs;
    const int total = num_kv_heads * bs * LANES;  // a multiple of 64: whole warps
    const int first = blockIdx.y * (kReadThreads * kReadDepth) + threadIdx.x;
    uint32_t word[kReadDepth], param[kReadDepth];
    const int j = (threadIdx.x % LANES) / 4, u = 2 * (threadIdx.x % 4);
    const bool odd = j & 1;
#pragma unroll
    for (int k = 0; k < kReadDepth; ++k) {
        const int i = first + k * kReadThreads;
        word[k] = param[k] = 0;
        if (i < total) {
            const int row = i / LANES;  // head * bs + offset
            const char *base = from + static_cast<int64_t>(row >> block_shift) * record;
            const int off = row & (bs - 1);
            word[k] = *reinterpret_cast<const uint32_t *>(base + off * (D / 2) + ((u + odd) * NG + (j & ~1)) * 2);
            param[k] = *reinterpret_cast<const uint32_t *>(base + bs * (D / 2) + off * (D / 8) + j * 4);
        }
    }
#pragma unroll
    for (int k = 0; k < kReadDepth; ++k) {
        const int i = first + k * kReadThreads;
        // this lane's word: unit u of groups j, j + 1 (j even) or unit u + 1 of groups j - 1, j
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word[k] & 0xffffu : word[k] >> 16, 4);
        const uint32_t codes = odd ? (other | (word[k] & 0xffff0000u)) : ((word[k] & 0xffffu) | (other << 16));
        const float2 sz = pkv::Int4Param<T>::unpack(param[k]);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = static_cast<float>((codes >> (8 * e)) & 15u), b = static_cast<float>((codes >> (8 * e + 4)) & 15u);
            w[e] = pkv::Elem<T>::pack2(fmaf(a, sz.x, sz.y), fmaf(b, sz.x, sz.y));
        }
        if (i < total) to[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

bool supported_shape(int head_dim, int block_size) {
    return (head_dim == 64 || head_dim == 128) && (block_size == 8 || block_size == 16 || block_size == 32);
}

int shift_of(int block_size) { return block_size == 8 ? 3 : block_size == 16 ? 4 : 5; }

}  // namespace

extern "C" {

PKV_API pkv_status pkv_reshape_and_cache_int4(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                                              int64_t num_tokens, void *k_cache, void *v_cache, int64_t num_blocks,
                                              int64_t block_stride_bytes, int num_kv_heads, int head_dim,
                                              int block_size, pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (!supported_shape(head_dim, block_size)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks <= 0 || num_tokens > 0x7fffff00LL / num_kv_heads)
        return PKV_ERR_INVALID_ARG;
    const int64_t half = static_cast<int64_t>(num_kv_heads) * pkv::int4_record_bytes(head_dim, block_size);
    if (block_stride_bytes < half || block_stride_bytes % 16) return PKV_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !slot_mapping || !pkv::aligned16(k_new) || !pkv::aligned16(v_new) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    const int64_t rows = num_tokens * num_kv_heads;
    const int per_cta = kWriteThreads / (head_dim / 8);
    auto kernel = dtype == PKV_F16 ? (head_dim == 128 ? reshape_and_cache_int4_kernel<__half, 128> : reshape_and_cache_int4_kernel<__half, 64>)
                                   : (head_dim == 128 ? reshape_and_cache_int4_kernel<__nv_bfloat16, 128>
                                                      : reshape_and_cache_int4_kernel<__nv_bfloat16, 64>);
    kernel<<<static_cast<unsigned>((rows + per_cta - 1) / per_cta), kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), slot_mapping, static_cast<char *>(k_cache),
        static_cast<char *>(v_cache), num_blocks * block_size, block_stride_bytes, static_cast<int>(rows), num_kv_heads,
        shift_of(block_size), status);
    pkv::count_launch();
    return pkv::launch_status();
}

PKV_API pkv_status pkv_dequantise_blocks_int4(const void *k_cache4, const void *v_cache4, int64_t num_blocks4,
                                              int64_t block_stride_bytes4, const int64_t *src_dst_pairs,
                                              int64_t num_pairs, void *k_cache, void *v_cache, int64_t num_blocks,
                                              int64_t block_stride_elems, int num_kv_heads, int head_dim,
                                              int block_size, pkv_dtype dtype, void *stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (!supported_shape(head_dim, block_size)) return PKV_ERR_UNSUPPORTED;
    if (num_pairs < 0 || num_pairs > 0x7fffffffLL || num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks4 <= 0 || num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    const int64_t half4 = static_cast<int64_t>(num_kv_heads) * pkv::int4_record_bytes(head_dim, block_size);
    const int64_t half = static_cast<int64_t>(num_kv_heads) * block_size * head_dim;
    if (block_stride_bytes4 < half4 || block_stride_bytes4 % 16 || block_stride_elems < half || block_stride_elems % 8)
        return PKV_ERR_INVALID_ARG;
    if (!k_cache4 || !v_cache4 || !k_cache || !v_cache || !pkv::aligned16(k_cache4) || !pkv::aligned16(v_cache4) ||
        !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return PKV_ERR_INVALID_ARG;
    if (num_pairs == 0) return PKV_OK;
    if (!src_dst_pairs || (reinterpret_cast<uintptr_t>(src_dst_pairs) & 7u)) return PKV_ERR_INVALID_ARG;
    unsigned int *status = pkv::status_word_ptr();
    if (!status) return PKV_ERR_CUDA;
    const int64_t chunks = (half / 8 + kReadThreads * kReadDepth - 1) / (kReadThreads * kReadDepth);
    if (chunks > 65535) return PKV_ERR_INVALID_ARG;
    auto kernel = dtype == PKV_F16 ? (head_dim == 128 ? dequantise_blocks_int4_kernel<__half, 128> : dequantise_blocks_int4_kernel<__half, 64>)
                                   : (head_dim == 128 ? dequantise_blocks_int4_kernel<__nv_bfloat16, 128>
                                                      : dequantise_blocks_int4_kernel<__nv_bfloat16, 64>);
    kernel<<<dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>(chunks), 2), kReadThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const char *>(k_cache4), static_cast<const char *>(v_cache4), num_blocks4, block_stride_bytes4,
        src_dst_pairs, static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), num_blocks, block_stride_elems / 8,
        num_kv_heads, shift_of(block_size), status);
    pkv::count_launch();
    return pkv::launch_status();
}

}  // extern "C"
