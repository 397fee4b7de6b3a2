// int4_cache.cu -- the 4-bit cache's write and read-back (format: int4.cuh):
//   pkv_reshape_and_cache_int4    quantise each new token's K/V rows into its slot
//   pkv_dequantise_blocks_int4    blocks of a 4-bit pool -> blocks of a 16-bit pool
// Both move a few bytes per value and are bound by memory: 2 + 5/8 bytes a value each way.  They are launched
// ahead, like the other short kernels that follow one another in a step, and wait for the kernel before them with
// their blocks in place (8192 tokens written and read back: 15.6 us one behind the other, 21.3 launched in the usual way).
#include <type_traits>

#include "int4.cuh"
#include "pkv_host.h"

namespace {

// The low half: a group's smallest value, the high half: its largest one's negative; 16 values in each of
// two lanes, packed in the rows' type.  A NaN among them comes through (kNan) or loses.
template <typename T, bool kNan>
__device__ __forceinline__ float2 int4_range(const uint4 (&row)[2]) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    auto least = [](T2 a, T2 b) { return kNan ? __hmin2_nan(a, b) : __hmin2(a, b); };
    auto most = [](T2 a, T2 b) { return kNan ? __hmax2_nan(a, b) : __hmax2(a, b); };
    const T2 *v = reinterpret_cast<const T2 *>(row);
    T2 lo = v[0], hi = v[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) lo = least(lo, v[e]), hi = most(hi, v[e]);
    T2 m;
    m.x = kNan ? __hmin_nan(lo.x, lo.y) : __hmin(lo.x, lo.y);
    m.y = __hneg(kNan ? __hmax_nan(hi.x, hi.y) : __hmax(hi.x, hi.y));
    const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&m), 1);
    m = least(m, *reinterpret_cast<const T2 *>(&other));
    return pkv::Int4Param<T>::unpack(*reinterpret_cast<const uint32_t *>(&m));
}

// The smallest scale with 15 s >= hi - lo, as bits: a number of the type that is surely not above it, then
// up while 15 s (exact) is too small.
template <typename T>
__device__ __forceinline__ uint32_t int4_scale(float lo, float hi) {
    const float range = __fsub_ru(hi, lo);
    uint32_t sb = pkv::Int4Param<T>::scale_down(range * 0.06666663f);
    if (15.f * pkv::Int4Param<T>::value(sb) < range) ++sb;
    if (15.f * pkv::Int4Param<T>::value(sb) < range) ++sb;
    return sb;
}

// Four codes, each in the low bits of a word whose other low bits are zero -> one 16-bit word, the first in
// its low nibble (the bits above are not cleared).
__device__ __forceinline__ uint32_t int4_word(const uint32_t *c) {
    return c[0] + 16u * c[1] + 256u * c[2] + 4096u * c[3];
}

// Quantises the 16 channels 16 i .. 16 i + 15 of a group whose two lanes call together: the 16-bit code
// words of its units 4 i .. 4 i + 3 in two registers, and the group's (s, z) word.
//
// A code is the quotient d / s, d = x - z in fp32, rounded to fp32 and then to an integer, ties to even.  The quotient
// comes from an approximate reciprocal, a remainder d - q s (exact in one FMA) and one correction, and is
// d / s (1 + 2^-46) before its rounding: a tie (k + 1/2) s = d gives k + 1/2 itself.  No other d rounds to a
// tie: s has 11 bits at most, so (k + 1/2) s is a fp32 number like d, and they differ by a step of d, which
// is more than half a step of fp32 at k + 1/2 by the factor 2 / m with the mantissa m <= 2 - 2^-10 of s.  Adding
// 1.5 * 2^23 rounds to an integer and leaves it in the low bits.
template <typename T>
__device__ __forceinline__ void int4_quantise(const uint4 (&row)[2], uint32_t (&unit)[2], uint32_t &param) {
    float2 r = int4_range<T, true>(row);
    uint32_t sb = int4_scale<T>(r.x, -r.y);
    float s = pkv::Int4Param<T>::value(sb), f[16];
    pkv::Elem<T>::to_f32x8(row[0], *reinterpret_cast<float(*)[8]>(f));
    pkv::Elem<T>::to_f32x8(row[1], *reinterpret_cast<float(*)[8]>(f + 8));
    uint32_t c[16];
    // 2^-100 <= s < 2^100 or 0; a scale whose reciprocal would overflow or vanish, infinite (a spread past fp32's range too)
    // or NaN, takes the division
    const bool in_range = s == 0.f || __float_as_uint(s) - 0x0d800000u < 0x64000000u;
    if (__all_sync(0xffffffffu, in_range)) {
        const float by = s == 0.f ? 0.f : pkv::fast_rcp(s);
        const pkv::F32x2 minus_z = pkv::pack_f32(-r.x, -r.x), rcp = pkv::pack_f32(by, by), minus_s = pkv::pack_f32(-s, -s),
                         round = pkv::pack_f32(12582912.f, 12582912.f);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const pkv::F32x2 d = pkv::add2(pkv::pack_f32(f[e], f[e + 1]), minus_z), q = pkv::mul2(d, rcp);
            const pkv::F32x2 t = pkv::add2(pkv::fma2(pkv::fma2(q, minus_s, d), rcp, q), round);
            float t0, t1;
            pkv::unpack_f32(t, t0, t1);
            c[e] = __float_as_uint(t0);
            c[e + 1] = __float_as_uint(t1);
        }
    } else {
        r = int4_range<T, false>(row);
        // a group that spreads over more than fp32 holds is taken by quarters (exact: its values are bf16)
        const float by = -r.y - r.x == INFINITY ? 0.25f : 1.f;
        sb = int4_scale<T>(r.x * by, -r.y * by);
        s = pkv::Int4Param<T>::value(sb);
#pragma unroll
        for (int e = 0; e < 16; ++e) c[e] = static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(f[e] * by - r.x * by, s)), 0.f), 15.f));
        if (by != 1.f) sb = pkv::Int4Param<T>::bits(4.f * s);
    }
    param = sb | (pkv::Int4Param<T>::bits(r.x) << 16);
    unit[0] = __byte_perm(int4_word(c), int4_word(c + 4), 0x5410);
    unit[1] = __byte_perm(int4_word(c + 8), int4_word(c + 12), 0x5410);
}

// A thread quantises 16 channels of one row of K and of V; the rows of a token and then the tokens follow one
// another.  Lanes 2 j + i hold channels 16 i .. of group j; the lanes of a row's groups trade words, so
// that each stores eight bytes side by side (all groups of a unit, or of two).  Bound by arithmetic:
// 8192 tokens of 8 heads of 128, bf16 8.0 us, 0.81 of measured HBM (with eight channels per lane and the remainder's comparison instead
// of the quotient's correction 15.3, with a division and a CTA per token 22).
constexpr int kWriteThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads) reshape_and_cache_int4_kernel(
    const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, const int64_t *__restrict__ slot_mapping,
    char *__restrict__ k_cache, char *__restrict__ v_cache, int64_t num_slots, int64_t block_stride, int num_rows,
    int num_kv_heads, pkv::FastDiv div_kv_heads, int block_shift, unsigned int *status) {
    constexpr int LANES = D / 16;
    pkv::pdl_trigger();
    pkv::pdl_wait();
    const int row = blockIdx.x * (kWriteThreads / LANES) + threadIdx.x / LANES;  // token * num_kv_heads + head
    const int lane = threadIdx.x % LANES, j = lane / 2, i = lane % 2;
    const bool there = row < num_rows;
    uint4 x[2][2] = {};
    int64_t slot = -1;
    const int n = pkv::fast_div(row, div_kv_heads), h = row - n * num_kv_heads;
    if (there) {
        const int64_t at = static_cast<int64_t>(row) * (D / 8) + 2 * lane;
        slot = slot_mapping[n];
        x[0][0] = k_new[at];
        x[0][1] = k_new[at + 1];
        x[1][0] = v_new[at];
        x[1][1] = v_new[at + 1];
    }
    if (slot >= num_slots) {
        if (h == 0 && lane == 0) pkv::raise_flag(status, PKV_DEVERR_SLOT);
        slot = -1;
    }
    const int bs = 1 << block_shift, off = static_cast<int>(slot) & (bs - 1);
    const int64_t at = (slot >> block_shift) * block_stride + static_cast<int64_t>(h) * pkv::int4_record_bytes(D, bs);
    const bool odd = j & 1, upper = j & 2;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t unit[2], param;
        int4_quantise<T>(x[half], unit, param);
        // units 4 i + 2 odd, + 1 of groups j & ~1, j | 1
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? unit[0] : unit[1], 2);
        const uint32_t even_group = odd ? other : unit[0], odd_group = odd ? unit[1] : other;
        uint2 w = make_uint2(__byte_perm(even_group, odd_group, 0x5410), __byte_perm(even_group, odd_group, 0x7632));
        int place = (4 * i + 2 * odd) * 4;
        if constexpr (D == 128) {
            // unit 4 i + 2 odd + upper of all groups
            const uint32_t from = __shfl_xor_sync(0xffffffffu, upper ? w.x : w.y, 4);
            w = upper ? make_uint2(from, w.y) : make_uint2(w.x, from);
            place = (4 * i + 2 * odd + upper) * 8;
        }
        if (slot >= 0) {
            char *base = (half ? v_cache : k_cache) + at;
            *reinterpret_cast<uint2 *>(base + off * (D / 2) + place) = w;
            if (i == 0) *reinterpret_cast<uint32_t *>(base + bs * (D / 2) + off * (D / 8) + j * 4) = param;
        }
    }
}

constexpr int kReadThreads = 256;
constexpr int kReadDepth = 4;  // vectors of a thread in flight

// grid.x = pair, grid.y = chunk of a half block's vectors, grid.z = K (0) / V (1); a
// thread writes 8 channels (16 bytes) of a row: lanes 4 j + i those of 8 i .. in group j.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) dequantise_blocks_int4_kernel(
    const char *__restrict__ k4, const char *__restrict__ v4, int64_t num_blocks4, int64_t block_stride4,
    const int64_t *__restrict__ pairs, uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache, int64_t num_blocks,
    int64_t block_stride_vecs, int num_kv_heads, int block_shift, unsigned int *status) {
    constexpr int LANES = D / 8, NG = D / 32;
    pkv::pdl_trigger();
    pkv::pdl_wait();
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
            w[e] = pkv::Int4Param<T>::pack2_finite(fmaf(a, sz.x, sz.y), fmaf(b, sz.x, sz.y));
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
    const int per_cta = kWriteThreads / (head_dim / 16);
    auto kernel = dtype == PKV_F16 ? (head_dim == 128 ? reshape_and_cache_int4_kernel<__half, 128> : reshape_and_cache_int4_kernel<__half, 64>)
                                   : (head_dim == 128 ? reshape_and_cache_int4_kernel<__nv_bfloat16, 128>
                                                      : reshape_and_cache_int4_kernel<__nv_bfloat16, 64>);
    if (pkv::launch_kernel(kernel, dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta)), dim3(kWriteThreads), 0,
                           static_cast<cudaStream_t>(stream), true, static_cast<const uint4 *>(k_new),
                           static_cast<const uint4 *>(v_new), slot_mapping, static_cast<char *>(k_cache),
                           static_cast<char *>(v_cache), num_blocks * block_size, block_stride_bytes, static_cast<int>(rows),
                           num_kv_heads, pkv::make_fast_div(num_kv_heads), shift_of(block_size), status) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
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
    if (pkv::launch_kernel(kernel, dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>(chunks), 2), dim3(kReadThreads), 0,
                           static_cast<cudaStream_t>(stream), true, static_cast<const char *>(k_cache4),
                           static_cast<const char *>(v_cache4), num_blocks4, block_stride_bytes4, src_dst_pairs,
                           static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), num_blocks, block_stride_elems / 8,
                           num_kv_heads, shift_of(block_size), status) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    pkv::count_launch();
    return pkv::launch_status();
}

}  // extern "C"
