// int4.cuh -- the 4-bit cache's row format, shared by its write, its read-back and its decode.
//
// A row of head_dim values of one token and KV head is cut into groups of 32 channels;
// group j holds a zero z (its smallest value), a scale s (the smallest value of the rows'
// type that is at least (max - min) / 15) and codes c in 0 .. 15 that stand for s c + z.
// z is one of the row's own values and s is rounded up, so every value lies in
// [z, z + 15 s] and no code saturates: a value is off by s / 2 at most.  z + 15 s itself may
// lie past the type's range, by less than s / 2: what is read back stops at its largest finite value.
//
// A block's record of one KV head holds the codes of its tokens, head_dim / 2 bytes each,
// then the (s, z) pairs of its tokens, head_dim / 32 of them each: 80 bytes a token at
// head_dim 128, one contiguous copy per block.  Channel 32 j + 4 u + e of a token is nibble e of
// its 16-bit word u * NG + j (NG = head_dim / 32 groups, u = 0 .. 7), so that a unit u (2 NG
// bytes) holds four channels of every group.  The decode's MMA fragments fall out of it: a
// lane's 16 (or 8) bytes of a K row are two units, and a byte permute of two units or two
// tokens pairs values of one group.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

__host__ __device__ constexpr int int4_row_bytes(int head_dim) { return head_dim / 2; }     // codes
__host__ __device__ constexpr int int4_param_bytes(int head_dim) { return head_dim / 8; }   // (s, z) pairs
__host__ __device__ constexpr int int4_record_bytes(int head_dim, int block_size) {
    return block_size * (int4_row_bytes(head_dim) + int4_param_bytes(head_dim));
}

template <typename T>
struct Int4Param;  // a (scale, zero) pair as one 32-bit word, the scale in the low half

template <>
struct Int4Param<__half> {
    static __device__ __forceinline__ uint32_t scale_down(float x) { return __half_as_ushort(__float2half_rd(x)); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __half_as_ushort(__float2half_rn(x)); }
    static __device__ __forceinline__ float value(uint32_t b) { return __half2float(__ushort_as_half(static_cast<unsigned short>(b))); }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    // two values rounded to the type, those past its range to its largest finite ones (NaN stays)
    static __device__ __forceinline__ uint32_t pack2_finite(float a, float b) {
        uint32_t d;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(a), "f"(b));
        return d;
    }
};

template <>
struct Int4Param<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t scale_down(float x) { return __bfloat16_as_ushort(__float2bfloat16_rd(x)); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
    static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack2_finite(float a, float b) {
        uint32_t d;
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(a), "f"(b));
        return d;
    }
};

}  // namespace pkv
