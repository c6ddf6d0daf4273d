// What the experts' products share: activations, bias, eight elements of a row,
// a scan over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_rows_kernels.hpp"

namespace mxq {

enum LinearAct { kActNone, kActRelu, kActGelu, kActSilu };

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int wave_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(v, d, 64);
        if (lane >= d)
            v += y;
    }
    return v;
}

// The normal distribution's cdf at x and e = exp(-x^2 / 2).  Its tail at z = |x| is
// e t P(t) with t = 1 / (1 + 0.3 z), as tail / e falls smoothly like 1 / z; P, of
// degree 7, has the least largest relative error for z from 0 to 14, 1.4e-7 (a
// linear program over 1200 values of t).  With the roundings to fp32 3e-7 absolute
// and, what GELU's values far below zero are made of, 6e-7 of the tail up to
// z = 3 and 1e-5 at 13, where the exponent's own rounding leaves no more: far under
// the rounding to bf16 in either sense.  16 instructions where erff takes 40:
// results pass here while the matrix units wait.
__device__ __forceinline__ void normal_cdf(float x, float &cdf, float &e)
{
    const float z = fabsf(x), t = __builtin_amdgcn_rcpf(fmaf(z, 0.3f, 1.0f));
    float p = fmaf(t, 0.035568062f, -0.15678892f);
    p = fmaf(t, p, 0.20569530f);
    p = fmaf(t, p, -0.053129558f);
    p = fmaf(t, p, 0.12829505f);
    p = fmaf(t, p, 0.099986769f);
    p = fmaf(t, p, 0.12074330f);
    p = fmaf(t, p, 0.11962993f);
    e = __builtin_amdgcn_exp2f(x * x * -0.72134752f);
    const float tail = t * p * e;
    cdf = x >= 0.0f ? 1.0f - tail : tail;
}

__device__ __forceinline__ float sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

__device__ __forceinline__ float act_value(int act, float x)
{
    if (act == kActRelu)
        return x < 0.0f ? 0.0f : x;  // a NaN stays one
    if (act == kActGelu) {
        float cdf, e;
        normal_cdf(x, cdf, e);
        return x * cdf;
    }
    if (act == kActSilu)
        return x * sigmoid(x);
    return x;
}

// eight values; one branch for all of them
__device__ __forceinline__ void act_values(int act, float (&v)[8])
{
    if (act == kActRelu) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = act_value(kActRelu, v[k]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = act_value(kActGelu, v[k]);
    } else if (act == kActSilu) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = act_value(kActSilu, v[k]);
    }
}

// act(x) and act'(x)
__device__ __forceinline__ void act_both(int act, float x, float &y, float &slope)
{
    y = x;
    slope = 1.0f;
    if (act == kActRelu) {
        y = act_value(kActRelu, x);
        slope = x > 0.0f ? 1.0f : 0.0f;
    } else if (act == kActGelu) {
        float cdf, e;
        normal_cdf(x, cdf, e);
        y = x * cdf;
        slope = fmaf(x * 0.39894228f, e, cdf);
    } else if (act == kActSilu) {
        const float s = sigmoid(x);
        y = x * s;
        slope = s * fmaf(x, 1.0f - s, 1.0f);
    }
}

__device__ __forceinline__ float bias_at(const void *bias, int f32, int64_t at)
{
    return f32 ? reinterpret_cast<const float *>(bias)[at]
               : Piece<uint16_t>::to_f32(reinterpret_cast<const uint16_t *>(bias)[at]);
}

// eight elements of bf16 from column c of a row of n, c < n
__device__ __forceinline__ Piece<uint16_t> load8(const uint16_t *row, int c, int n)
{
    if (c + 8 <= n)
        return ld_piece<uint16_t>(row + c);
    Piece<uint16_t> r;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        r.v[k] = c + k < n ? row[c + k] : (uint16_t)0;
    return r;
}

__device__ __forceinline__ void store8(uint16_t *row, int c, int n, const float (&v)[8])
{
    Piece<uint16_t> r;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        r.set(k, v[k]);
    if (c + 8 <= n) {
        st_piece<uint16_t>(row + c, r);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < n)
            row[c + k] = r.v[k];
}

}  // namespace mxq
