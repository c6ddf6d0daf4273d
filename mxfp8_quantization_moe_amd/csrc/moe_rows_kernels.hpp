// Token rows into expert groups and back: dispatch, combine and their
// gradients.
//
// A token t has k slots; slot (t, j) names row r = rows[t*k + j] of a buffer
// of `capacity` rows laid out group after group (a row outside [0, capacity)
// is an empty slot).
//   dispatch          out[r] = x_t                    (and zeros elsewhere)
//   combine           y_t = resid_t + sum_j w_tj in[r], j ascending, fp32,
//                     rounded once
//   combine backward  out[r] = w_tj dy_t (and zeros elsewhere),
//                     dw_tj = sum_c dy_tc in[r]_c in fp32
// Everything is bound by memory.  Every kernel works from the token side, so
// a token's row moves once however many slots it has, and each expert-side
// row moves once by construction: no atomics, and a sum's order is fixed by
// the slot order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_device.hpp"

namespace mxq {

constexpr int kRowsThreads = 256;

// 16 bytes of a row as fp32 values.  Rows start on any element, so the
// vector type promises no more alignment than the element's (global memory
// instructions take any alignment on gfx950).
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
    static constexpr int N = 8;
    typedef uint16_t V __attribute__((ext_vector_type(8), aligned(2)));
    V v;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float((uint32_t)v[i] << 16); }
    __device__ __forceinline__ void set(int i, float f) { v[i] = from_f32(f); }
    // round to nearest even; a NaN keeps its sign and top bits and stays a NaN
    static __device__ __forceinline__ uint16_t from_f32(float f)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    }
    static __device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
};
template <>
struct Piece<float> {
    static constexpr int N = 4;
    typedef float V __attribute__((ext_vector_type(4), aligned(4)));
    V v;
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ void set(int i, float f) { v[i] = f; }
    static __device__ __forceinline__ float from_f32(float f) { return f; }
    static __device__ __forceinline__ float to_f32(float f) { return f; }
};

// Start of piece p of a row of `width` >= N elements: the last piece is moved
// back to end with the row.  Its overlap with the piece before it is loaded
// and stored twice with equal values, so no row needs an element-wise tail.
template <typename T>
__device__ __forceinline__ int piece_start(int p, int width)
{
    const int c = p * Piece<T>::N;
    return c + Piece<T>::N <= width ? c : width - Piece<T>::N;
}

// STREAM: with the nontemporal hint, for calls that move more than the caches
// hold.  Three sets of inputs in turn, one call after the other: 16384 tokens
// of 4096 bf16 over 2 slots (402 MB) dispatch 75 -> 61 us, combine 71 -> 62, its
// gradient 132 -> 105; 8192 tokens 33.3 -> 33.3, 34.0 -> 34.6, 69 -> 57; 4096
// tokens (100 MB) lose: 16.9 -> 19.5, 16.4 -> 18.4, 30.8 -> 30.0.  Dispatch and
// its gradient in turn 153 -> 144, combine and its gradient 190 -> 186.  The
// hint on the stores as well, or on them alone, is slower (70 and 72 us for
// the first).
template <typename T, bool STREAM = false>
__device__ __forceinline__ Piece<T> ld_piece(const T *p)
{
    Piece<T> r;
    if constexpr (STREAM)
        r.v = __builtin_nontemporal_load(reinterpret_cast<const typename Piece<T>::V *>(p));
    else
        r.v = *reinterpret_cast<const typename Piece<T>::V *>(p);
    return r;
}
template <typename T>
__device__ __forceinline__ void st_piece(T *p, const Piece<T> &v)
{
    *reinterpret_cast<typename Piece<T>::V *>(p) = v.v;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The rows no slot names: the padding of each group, [end of its rows, offs),
// and everything past the last group.  Workgroup z of nz takes every nz-th
// group's padding and every nz-th row of the tail.  Offsets are clamped to
// the buffer.  Eight groups of 16384 tokens of 4096 bf16: dispatch 62 us with
// up to 15 rows of padding each, 74 with up to 127, 215 with up to 1023.
template <typename T>
__device__ __forceinline__ void zero_rows(int z, int nz, const int32_t *__restrict__ counts,
                                          const int32_t *__restrict__ offs, int experts, T *out, int64_t ld,
                                          int capacity, int width)
{
    auto clear = [&](int64_t r) {
        T *row = out + r * ld;
        if (width < Piece<T>::N) {
            for (int c = threadIdx.x; c < width; c += kRowsThreads)
                row[c] = 0;
            return;
        }
        Piece<T> zero;
#pragma unroll
        for (int i = 0; i < Piece<T>::N; ++i)
            zero.v[i] = 0;
        const int pieces = (width + Piece<T>::N - 1) / Piece<T>::N;
        for (int p = threadIdx.x; p < pieces; p += kRowsThreads)
            st_piece<T>(row + piece_start<T>(p, width), zero);
    };
    for (int e = z; e < experts; e += nz) {
        const int64_t start = e ? min(max(offs[e - 1], 0), capacity) : 0;
        const int end = min(max(offs[e], 0), capacity);
        for (int64_t r = start + max(counts[e], 0); r < end; ++r)
            clear(r);
    }
    const int tail = min(max(offs[experts - 1], 0), capacity);
    for (int64_t r = tail + z; r < capacity; r += nz)
        clear(r);
}

// One wave per (token, chunk of 64 * U pieces); the workgroups past
// `work` blocks clear the rows without a slot.  16384 tokens of 4096 bf16 over
// 2 slots: 61 us for 403 MB (6.6 TB/s) after calls of its own kind, 74 (5.4)
// after its gradient on other rows: bound by memory.
template <typename T, int U, bool STREAM>
__global__ __launch_bounds__(kRowsThreads) void moe_dispatch_kernel(
    const T *__restrict__ x, int64_t sx, int tokens, int width, const int32_t *__restrict__ rows, int k,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offs, int experts, T *__restrict__ out,
    int64_t ld, int capacity, int chunks, int work)
{
    constexpr int N = Piece<T>::N;
    if ((int)blockIdx.x >= work) {
        zero_rows<T>(blockIdx.x - work, gridDim.x - work, counts, offs, experts, out, ld, capacity, width);
        return;
    }
    const int lane = threadIdx.x & 63;
    const int64_t item = uniform(blockIdx.x * (kRowsThreads / 64) + (threadIdx.x >> 6));
    const int t = (int)(item / chunks), chunk = (int)(item % chunks);
    if (t >= tokens)
        return;
    const T *src = x + (int64_t)t * sx;
    const int32_t *slots = rows + (int64_t)t * k;
    if (width < N) {
        for (int j = 0; j < k; ++j) {
            const int r = slots[j];
            if (r >= 0 && r < capacity && lane < width)
                out[(int64_t)r * ld + lane] = src[lane];
        }
        return;
    }
    const int pieces = (width + N - 1) / N, p0 = chunk * 64 * U + lane;
    Piece<T> v[U];
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        c[u] = piece_start<T>(min(p0 + 64 * u, pieces - 1), width);
        v[u] = ld_piece<T, STREAM>(src + c[u]);
    }
    for (int j = 0; j < k; ++j) {
        const int r = slots[j];
        if (r < 0 || r >= capacity)
            continue;
        T *dst = out + (int64_t)r * ld;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p0 + 64 * u < pieces)
                st_piece<T>(dst + c[u], v[u]);
    }
}

// One wave per (token, chunk of 64 pieces), KB slots' loads in flight at a
// time.  Loads of empty slots go to row 0 and are not used.  More pieces per
// lane make fewer, longer waves, which is slower: 16384 tokens of 2048 bf16
// over 2 slots 32.6 us, 36.7 with four; of 4096 62.8 us, 66.3.  Between other
// passes, its rows in no cache, the last takes 72 us (5.6 TB/s); 8 tokens of
// 5120 over 8 slots 3.7 us.  Slots that do not fill a block of KB cost little:
// rows of 4096 bf16 over 1, 3, 5 and 9 slots run at 5.9, 6.3, 5.9 and 5.4 TB/s,
// over 2, 4, 8 and 16 at 6.4, 6.1, 5.8 and 5.7.
template <typename T, int KB, bool STREAM>
__global__ __launch_bounds__(kRowsThreads) void moe_combine_kernel(
    const T *__restrict__ in, int64_t ld, int capacity, int width, const int32_t *__restrict__ rows,
    const float *__restrict__ weights, int k, const T *__restrict__ resid, int64_t sr, T *__restrict__ y,
    int64_t sy, int tokens, int chunks)
{
    constexpr int N = Piece<T>::N;
    const int lane = threadIdx.x & 63;
    const int64_t item = uniform(blockIdx.x * (kRowsThreads / 64) + (threadIdx.x >> 6));
    const int t = (int)(item / chunks), chunk = (int)(item % chunks);
    if (t >= tokens)
        return;
    const int32_t *slots = rows + (int64_t)t * k;
    const float *wt = weights ? weights + (int64_t)t * k : nullptr;
    if (width < N) {
        if (lane >= width)
            return;
        float s = resid ? Piece<T>::to_f32(resid[(int64_t)t * sr + lane]) : 0.0f;
        for (int j = 0; j < k; ++j) {
            const int r = slots[j];
            if (r >= 0 && r < capacity)
                s = fmaf(wt ? wt[j] : 1.0f, Piece<T>::to_f32(in[(int64_t)r * ld + lane]), s);
        }
        y[(int64_t)t * sy + lane] = Piece<T>::from_f32(s);
        return;
    }
    const int pieces = (width + N - 1) / N, p = chunk * 64 + lane;
    const int c = piece_start<T>(min(p, pieces - 1), width);
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = 0.0f;
    if (resid) {
        const Piece<T> v = ld_piece<T, STREAM>(resid + (int64_t)t * sr + c);
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[i] = v.get(i);
    }
    for (int j0 = 0; j0 < k; j0 += KB) {
        Piece<T> v[KB];
        int r[KB];
        float w[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int jj = min(j0 + j, k - 1);
            r[j] = slots[jj];
            w[j] = wt ? wt[jj] : 1.0f;
            if (j0 + j >= k || r[j] < 0 || r[j] >= capacity)
                r[j] = -1;
            v[j] = ld_piece<T, STREAM>(in + (int64_t)max(r[j], 0) * ld + c);
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (r[j] < 0)
                continue;
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] = fmaf(w[j], v[j].get(i), acc[i]);
        }
    }
    Piece<T> o;
#pragma unroll
    for (int i = 0; i < N; ++i)
        o.set(i, acc[i]);
    if (p < pieces)
        st_piece<T>(y + (int64_t)t * sy + c, o);
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

// NW waves per token; each lane holds its piece of dy while KB slots' rows
// pass, and the dot products meet in a fixed order (lane tree, then waves).
// 16384 tokens of 4096 bf16 over 2 slots, a tenth masked: 122 us for 652 MB
// (5.3 TB/s), bound by memory.  Rows of 4096 bf16 over 1, 3, 5 and 9 slots: 6.0,
// 6.1, 6.1 and 5.1 TB/s, over 2, 4, 8 and 16 6.4, 6.1, 6.1 and 5.8.
template <typename T, int NW, int KB, bool STREAM>
__global__ __launch_bounds__(kRowsThreads) void moe_combine_backward_kernel(
    const T *__restrict__ dy, int64_t sy, int tokens, int width, const T *__restrict__ in, int64_t ld,
    const int32_t *__restrict__ rows, const float *__restrict__ weights, int k,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offs, int experts, int capacity,
    T *__restrict__ out, int64_t ldo, float *__restrict__ dw, int work)
{
    constexpr int N = Piece<T>::N;
    constexpr int TPB = kRowsThreads / 64 / NW;  // tokens per workgroup
    __shared__ float part[NW > 1 ? KB * NW : 1];
    if ((int)blockIdx.x >= work) {
        zero_rows<T>(blockIdx.x - work, gridDim.x - work, counts, offs, experts, out, ldo, capacity, width);
        return;
    }
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x * TPB + wave / NW, wt = wave % NW;
    if (t >= tokens)  // only with one wave per token, where no wave waits for another
        return;
    const int32_t *slots = rows + (int64_t)t * k;
    const float *w = weights + (int64_t)t * k;
    const T *g = dy + (int64_t)t * sy;
    const int pieces = (width + N - 1) / N;
    for (int j0 = 0; j0 < k; j0 += KB) {
        int r[KB];
        float wj[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int jj = min(j0 + j, k - 1);
            r[j] = slots[jj];
            wj[j] = w[jj];
            dot[j] = 0.0f;
            if (j0 + j >= k || r[j] < 0 || r[j] >= capacity)
                r[j] = -1;
        }
        if (width < N) {
            if (lane < width && wt == 0) {
                const float d = Piece<T>::to_f32(g[lane]);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (r[j] < 0)
                        continue;
                    dot[j] = d * Piece<T>::to_f32(in[(int64_t)r[j] * ld + lane]);
                    out[(int64_t)r[j] * ldo + lane] = Piece<T>::from_f32(wj[j] * d);
                }
            }
        } else {
            for (int p = wt * 64 + lane; p < pieces; p += NW * 64) {
                const int c = piece_start<T>(p, width);
                const int skip = p * N - c;  // elements that the piece before has
                const Piece<T> d = ld_piece<T, STREAM>(g + c);
                Piece<T> v[KB];
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    v[j] = ld_piece<T, STREAM>(in + (int64_t)max(r[j], 0) * ld + c);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (r[j] < 0)
                        continue;
                    Piece<T> o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float di = d.get(i);
                        dot[j] = i >= skip ? fmaf(di, v[j].get(i), dot[j]) : dot[j];
                        o.set(i, wj[j] * di);
                    }
                    st_piece<T>(out + (int64_t)r[j] * ldo + c, o);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
            dot[j] = wave_sum(dot[j]);
        if constexpr (NW == 1) {
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (lane == j && j0 + j < k)
                    dw[(int64_t)t * k + j0 + j] = r[j] < 0 ? 0.0f : dot[j];
        } else {
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    part[j * NW + wt] = r[j] < 0 ? 0.0f : dot[j];
            __syncthreads();
            if ((int)threadIdx.x < KB && j0 + (int)threadIdx.x < k) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    s += part[threadIdx.x * NW + i];
                dw[(int64_t)t * k + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

}  // namespace mxq
