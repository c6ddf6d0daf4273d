// Weights straight from memory into the registers of a matrix instruction, for
// products of few rows: 16 rows of weights against 16 tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_ops.hpp"

namespace mxq {

// Steps of a sum, 16 rows of weights and 16 tokens each.
//   bf16  32 values: lane 16 q + i holds values 8 q .. 8 q + 7 of row i
//   MX    64 values: lane 16 q + i holds values 16 q .. 16 q + 15 of row i, one
//         16-byte load, and takes them as two steps of 32 (the order of a sum
//         is free as long as weights and tokens agree); e4m3 times a power of
//         two is exact in bf16
template <bool MX>
struct WeightStep;

template <>
struct WeightStep<false> {
    static constexpr int K = 32, PIECES = 1;
    Piece<uint16_t> v;
    __device__ __forceinline__ void load(const void *row, const uint8_t *, int k)
    {
        v = ld_piece<uint16_t>(reinterpret_cast<const uint16_t *>(row) + k + ((threadIdx.x & 63) >> 4) * 8);
    }
    __device__ __forceinline__ void load_tail(const void *row, const uint8_t *, int k, int end)
    {
        const int c = k + ((threadIdx.x & 63) >> 4) * 8;
        v = load8(reinterpret_cast<const uint16_t *>(row), min(c, end), end);
    }
    __device__ __forceinline__ bf16x8 piece(int) const { return __builtin_bit_cast(bf16x8, v.v); }
};

template <>
struct WeightStep<true> {
    static constexpr int K = 64, PIECES = 2;
    uint4 v;
    float scale;
    __device__ __forceinline__ void load(const void *row, const uint8_t *scales, int k)
    {
        const int c = k + ((threadIdx.x & 63) >> 4) * 16;
        v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(row) + c);
        scale = __uint_as_float((uint32_t)scales[c >> 5] << 23);
    }
    __device__ __forceinline__ void load_tail(const void *row, const uint8_t *scales, int k, int end)
    {
        v = make_uint4(0, 0, 0, 0);
        scale = 1.0f;
        if (k + (int)((threadIdx.x & 63) >> 4) * 16 < end)
            load(row, scales, k);
    }
    __device__ __forceinline__ bf16x8 piece(int h) const
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        struct Four {
            bf16x2 p[4];
        } r;
        const uint32_t a = h ? v.z : v.x, b = h ? v.w : v.y;
        r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
        r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
        r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
        r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
        return __builtin_bit_cast(bf16x8, r);
    }
};

// the tokens' values for piece h of a step, zeros past `end`
template <bool MX>
__device__ __forceinline__ bf16x8 token_piece(const uint16_t *row, int k, int h)
{
    const int q = (threadIdx.x & 63) >> 4, c = MX ? k + q * 16 + h * 8 : k + q * 8;
    return __builtin_bit_cast(bf16x8, ld_piece<uint16_t>(row + c).v);
}
template <bool MX>
__device__ __forceinline__ bf16x8 token_piece_tail(const uint16_t *row, int k, int h, int end)
{
    const int q = (threadIdx.x & 63) >> 4, c = MX ? k + q * 16 + h * 8 : k + q * 8;
    return __builtin_bit_cast(bf16x8, load8(row, min(c, end), end).v);
}

__device__ __forceinline__ bf16x8 zero_piece() { return __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0)); }

// Both sides in MXFP8: 128 values by the scaled instruction.  Lane 16 q + i holds
// bytes 16 q and 64 + 16 q on of row i and supplies the scale of its block q.
typedef int int8v __attribute__((ext_vector_type(8)));

// Zeros past `end`, a multiple of 32, and without `there`.
__device__ __forceinline__ int8v scaled_values(const uint8_t *row, int k, int end, bool there)
{
    const int c = k + ((threadIdx.x & 63) >> 4) * 16;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (there && c < end)
        a = *reinterpret_cast<const uint4 *>(row + c);
    if (there && c + 64 < end)
        b = *reinterpret_cast<const uint4 *>(row + c + 64);
    return int8v{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
__device__ __forceinline__ int scaled_scale(const uint8_t *scales, int64_t sb, int k, int end, bool there)
{
    const int q = (threadIdx.x & 63) >> 4;
    return there && k + q * 32 < end ? scales[(k / 32 + q) * sb] : 0;
}

}  // namespace mxq
