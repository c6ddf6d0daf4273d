// Newton-Schulz orthogonalisation of weight updates (the Muon optimiser's
// step on expert weights), on the matrix cores.
//
// Per matrix, X of m <= n (a tall matrix is taken transposed):
//   X = G / (|G|_F + eps);  `steps` times:  A = X X^T,  B = bA + cA^2,
//   X = aX + BX;            out = scale * X.
//
// Three products per step.  A and A^2 are symmetric: only the tiles on and
// below the diagonal are computed, each stored a second time mirrored.
//
// Numerics.  The products run on f16 MFMA with fp32 accumulators.  f16 keeps
// 11 bits; X, A and B have magnitudes known from the iteration (|X|_2 <= 1.3
// for the usual coefficients), so fixed powers of two (kScaleX, kScaleA,
// kScaleB) keep them far from f16's ends.  Rounding the operands alone would
// cost 1.4e-3 to 3e-3 of the result (relative 2-norm, simulated), more than
// the final bf16 rounding (1.65e-3).  Two exact rearrangements bring it to
// 3e-4 to 7e-4 without another product:
//   - X is carried in two f16 parts (22 bits), and a X + diag(B) X is added in
//     fp32 from both parts; only the product with the rest of B sees the high
//     part alone;
//   - the diagonals d of A and of B, which are the large entries when the
//     singular values are near one another, never enter an f16 operand: with
//     A = diag(d) + O,  A^2 = O O + d_i O_ij + O_ij d_j + diag(d^2), and the
//     last three terms are fp32 in the epilogue (O there from two f16 parts).
//
// Layout.  Every operand of a product is stored with the summed dim
// contiguous (X row-major for X X^T, X transposed for B X), padded with zeros
// to whole tiles, so the products need no bounds checks: padding rows of X
// stay zero through the iteration.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "mxq_device.hpp"

namespace mxq {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr float kScaleX = 8192.0f;   // |x| <= 1.3: up to 10650; room to 8
constexpr float kScaleA = 2048.0f;   // |o| <= 1.7; room to 32
constexpr float kScaleB = 2048.0f;   // |b| <= 3; room to 32
constexpr float kLow = 2048.0f;      // the low parts are stored times 2^11
constexpr int kBK = 64;              // summed elements per LDS tile: 128-byte rows
constexpr int kNormParts = 64;       // partial sums of a matrix's squared norm

// Buffers of one call; matrix e's parts are `e` strides further.
struct MuonBuffers {
    _Float16 *xh, *xl;      // [mp][np] high and low parts of X
    _Float16 *xt[2];        // [np][mp] the high part transposed, this step's and the next
    _Float16 *oh, *ol, *bo; // [mp][mp] off-diagonal A (two parts) and B
    float *d, *db;          // [mp] diagonals of A and B
    double *part;           // [kNormParts] partial sums of squares
    int mp, np;             // padded extents
};

struct MuonView {           // x(i, j) = p[e * se + i * si + j * sj], i < m, j < n
    int64_t se, si, sj;
    int m, n;
};

__device__ __forceinline__ void split_half(float v, _Float16 &hi, _Float16 &lo)
{
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * kLow);
}

__device__ __forceinline__ float join_half(_Float16 hi, _Float16 lo) { return (float)hi + (float)lo * (1.0f / kLow); }

// ---------------------------------------------------------------- norm, load

template <typename T>
__device__ __forceinline__ float muon_elem(const T *p)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)*p << 16);
    else
        return *p;
}

// Squares in fp64: no value of a finite bf16 or fp32 matrix over- or
// underflows, and the rate does not matter beside the reads.
template <typename T>
__global__ __launch_bounds__(256) void muon_norm_kernel(const T *__restrict__ g, MuonView v, double *part)
{
    __shared__ double sums[256];
    const int e = blockIdx.y;
    const T *p = g + e * v.se;
    // along the unit-stride dim
    const bool inner_j = v.sj == 1;
    const int64_t inner = inner_j ? v.n : v.m, outer = inner_j ? v.m : v.n, so = inner_j ? v.si : v.sj;
    const int64_t sin = inner_j ? v.sj : v.si;
    double s = 0.0;
    const int64_t total = inner * outer;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < total; k += (int64_t)kNormParts * 256) {
        const int64_t o = k / inner, i = k % inner;
        const double x = (double)muon_elem<T>(p + o * so + i * sin);
        s += x * x;
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int m = 128; m > 0; m >>= 1) {
        if ((int)threadIdx.x < m)
            sums[threadIdx.x] += sums[threadIdx.x + m];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        part[(int64_t)e * kNormParts + blockIdx.x] = sums[0];
}

// X = G / (norm + eps) into the padded buffers, 64 x 64 elements per
// workgroup through LDS, so that both layouts are written in rows.
template <typename T>
__global__ __launch_bounds__(256) void muon_load_kernel(const T *__restrict__ g, MuonView v, MuonBuffers b, float eps)
{
    __shared__ float tile[64][65];
    const int e = blockIdx.z, i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    double s = 0.0;
    for (int k = 0; k < kNormParts; ++k)
        s += b.part[(int64_t)e * kNormParts + k];
    // in fp64: the reciprocal of a tiny norm overflows fp32
    const double mul = (double)kScaleX / (sqrt(s) + (double)eps);
    const T *p = g + e * v.se;
    const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
    const bool inner_j = v.sj == 1;
    for (int r = row; r < 64; r += 4) {
        const int i = inner_j ? r : lane, j = inner_j ? lane : r;
        float x = 0.0f;
        if (i0 + i < v.m && j0 + j < v.n)
            x = (float)((double)muon_elem<T>(p + (i0 + i) * v.si + (j0 + j) * v.sj) * mul);
        tile[i][j] = x;
    }
    __syncthreads();
    const int64_t xo = (int64_t)e * b.mp * b.np;
    for (int r = row; r < 64; r += 4) {
        _Float16 hi, lo;
        split_half(tile[r][lane], hi, lo);
        b.xh[xo + (int64_t)(i0 + r) * b.np + j0 + lane] = hi;
        b.xl[xo + (int64_t)(i0 + r) * b.np + j0 + lane] = lo;
        split_half(tile[lane][r], hi, lo);
        b.xt[0][xo + (int64_t)(j0 + r) * b.mp + i0 + lane] = hi;
    }
}

// ---------------------------------------------------------------- products

// 16 bytes per lane from global memory straight into LDS: lane l's bytes go to
// lds + 16 l (lds wave-uniform).  The waits are explicit (wait_tiles).
__device__ __forceinline__ void load_lds16(const void *src, uint32_t lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)(uintptr_t)lds, 16, 0, 0);
}

// This wave's loads into LDS have landed and its LDS reads have returned;
// then the workgroup meets.
__device__ __forceinline__ void wait_tiles()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\t"
                 "s_barrier"
                 :
                 :
                 : "memory");
}

enum MuonMode { kModeA, kModeB, kModeX, kModeOut };

struct MuonStep {
    float a, b, c, out_scale;
    int cur;  // which xt holds X now
};

// C[i][j] = sum_k P[i][k] Q[j][k] on TM x TN tiles, WM x WN waves.
//   kModeA  P = Q = X (K = np): off-diagonal A in two parts, diagonal d
//   kModeB  P = Q = O (K = mp): off-diagonal B, diagonal db
//   kModeX  P = B, Q = X^T (K = mp): the next X in its three forms
//   kModeOut  the same, written to the caller's output instead
template <int MODE, int TM, int TN, int WM, int WN, typename TO = uint16_t>
__global__ __launch_bounds__(WM *WN * 64) void muon_product_kernel(MuonBuffers b, MuonStep st, TO *out, MuonView ov)
{
    constexpr int THREADS = WM * WN * 64;
    constexpr bool SYM = MODE == kModeA || MODE == kModeB;
    constexpr int FM = TM / WM / 16, FN = TN / WN / 16;  // 16 x 16 fragments of a wave
    constexpr int STAGE = (TM + TN) * kBK;               // f16 elements of one LDS stage
    static_assert(!SYM || TM == TN, "symmetric products use square tiles");
    __shared__ _Float16 lds[2 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // tile of this workgroup.  Workgroups go to the 8 XCDs in turn: give each
    // XCD a contiguous run of tiles, so neighbours share operand rows in its L2
    const int total = gridDim.x, xcd = blockIdx.x & 7, per = total >> 3, rem = total & 7;
    const int id = xcd * per + min(xcd, rem) + (blockIdx.x >> 3);
    const int tm = b.mp / TM, tn = SYM ? tm : b.np / TN;
    const int per_matrix = SYM ? tm * (tm + 1) / 2 : tm * tn;
    const int e = id / per_matrix;
    int t = id % per_matrix, bi, bj;
    if (SYM) {
        bi = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
        while ((bi + 1) * (bi + 2) / 2 <= t)
            ++bi;
        while (bi * (bi + 1) / 2 > t)
            --bi;
        bj = t - bi * (bi + 1) / 2;
    } else {
        bi = t % tm;
        bj = t / tm;
    }
    const int64_t xo = (int64_t)e * b.mp * b.np, ao = (int64_t)e * b.mp * b.mp;
    const int K = MODE == kModeA ? b.np : b.mp;
    const _Float16 *P, *Q;
    if (MODE == kModeA)
        P = Q = b.xh + xo;
    else if (MODE == kModeB)
        P = Q = b.oh + ao;
    else {
        P = b.bo + ao;
        Q = b.xt[st.cur] + xo;
    }
    P += (int64_t)bi * TM * K;
    Q += (int64_t)bj * TN * K;

    // A stage holds TM rows of P, then TN rows of Q, 64 elements (8 chunks of
    // 16 bytes) each; chunk c of row r lies at chunk c ^ ((r >> 1) & 7), so
    // that the 16 rows a fragment read touches fall on different banks.  The
    // loads into LDS are linear; the swizzle is in the address they read.
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)lds;
    auto load_stage = [&](int kt, int s) {
#pragma unroll
        for (int u = 0; u < (TM + TN) * 8 / THREADS; ++u) {
            const int slot = u * THREADS + tid;          // 16-byte slot of the stage
            const int r = slot >> 3, c = (slot & 7) ^ ((r >> 1) & 7);
            const _Float16 *src = r < TM ? P + (int64_t)r * K : Q + (int64_t)(r - TM) * K;
            const uint32_t dst = lds0 + (uint32_t)(s * STAGE * 2 + (u * THREADS + wave * 64) * 16);
            load_lds16(src + kt * kBK + c * 8, __builtin_amdgcn_readfirstlane(dst));
        }
    };

    float4v acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};

    const int kt_end = K / kBK;
    const int fr = lane & 15, fk = lane >> 4;
    load_stage(0, 0);
    wait_tiles();
    for (int kt = 0; kt < kt_end; ++kt) {
        if (kt + 1 < kt_end)
            load_stage(kt + 1, (kt + 1) & 1);
        const _Float16 *base = lds + (kt & 1) * STAGE;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            half8 pf[FM], qf[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int r = wm * FM * 16 + i * 16 + fr;
                pf[i] = *reinterpret_cast<const half8 *>(base + r * kBK + (((ks * 4 + fk) ^ ((r >> 1) & 7)) * 8));
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int r = TM + wn * FN * 16 + j * 16 + fr;
                qf[j] = *reinterpret_cast<const half8 *>(base + r * kBK + (((ks * 4 + fk) ^ ((r >> 1) & 7)) * 8));
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pf[i], qf[j], acc[i][j], 0, 0, 0);
        }
        wait_tiles();
    }

    // lane l holds rows 4 (l / 16) + 0..3 of column l % 16 of each fragment
    const int gi0 = bi * TM + wm * FM * 16 + 4 * fk, gj0 = bj * TN + wn * FN * 16 + fr;
    const bool mirror = SYM && bi != bj;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int gi = gi0 + 16 * i, gj = gj0 + 16 * j;
            if constexpr (MODE == kModeA) {
                half4 hi, lo;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = acc[i][j][r] * (1.0f / (kScaleX * kScaleX));
                    const bool diag = gi + r == gj;
                    if (diag)
                        b.d[(int64_t)e * b.mp + gj] = v;
                    _Float16 h, l;
                    split_half(diag ? 0.0f : v * kScaleA, h, l);
                    hi[r] = h;
                    lo[r] = l;
                    b.oh[ao + (int64_t)(gi + r) * b.mp + gj] = h;
                    b.ol[ao + (int64_t)(gi + r) * b.mp + gj] = l;
                }
                if (mirror) {
                    *reinterpret_cast<half4 *>(b.oh + ao + (int64_t)gj * b.mp + gi) = hi;
                    *reinterpret_cast<half4 *>(b.ol + ao + (int64_t)gj * b.mp + gi) = lo;
                }
            } else if constexpr (MODE == kModeB) {
                const float *d = b.d + (int64_t)e * b.mp;
                // O is symmetric: its (gj, gi..gi+3) entries are contiguous
                const half4 oh = *reinterpret_cast<const half4 *>(b.oh + ao + (int64_t)gj * b.mp + gi);
                const half4 ol = *reinterpret_cast<const half4 *>(b.ol + ao + (int64_t)gj * b.mp + gi);
                const float dj = d[gj];
                half4 h4;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float oo = acc[i][j][r] * (1.0f / (kScaleA * kScaleA));
                    const float o = join_half(oh[r], ol[r]) * (1.0f / kScaleA);
                    const bool diag = gi + r == gj;
                    const float di = d[gi + r];
                    const float aij = diag ? di : o;
                    const float a2 = oo + (diag ? di * di : (di + dj) * o);
                    const float v = st.b * aij + st.c * a2;
                    if (diag)
                        b.db[(int64_t)e * b.mp + gj] = v;
                    h4[r] = (_Float16)(diag ? 0.0f : v * kScaleB);
                    b.bo[ao + (int64_t)(gi + r) * b.mp + gj] = h4[r];
                }
                if (mirror)
                    *reinterpret_cast<half4 *>(b.bo + ao + (int64_t)gj * b.mp + gi) = h4;
            } else {
                const float *db = b.db + (int64_t)e * b.mp;
                half4 h4;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t at = xo + (int64_t)(gi + r) * b.np + gj;
                    const float x = join_half(b.xh[at], b.xl[at]);
                    const float v = (st.a + db[gi + r]) * x + acc[i][j][r] * (1.0f / kScaleB);
                    if constexpr (MODE == kModeX) {
                        _Float16 h, l;
                        split_half(v, h, l);
                        h4[r] = h;
                        b.xh[at] = h;
                        b.xl[at] = l;
                    } else if (gi + r < ov.m && gj < ov.n) {
                        const float o = v * st.out_scale;
                        out[e * ov.se + (int64_t)(gi + r) * ov.si + (int64_t)gj * ov.sj] =
                            __builtin_bit_cast(uint16_t, (__bf16)o);
                    }
                }
                if constexpr (MODE == kModeX)
                    *reinterpret_cast<half4 *>(b.xt[st.cur ^ 1] + xo + (int64_t)gj * b.mp + gi) = h4;
            }
        }
}

// With no steps the result is scale * X itself.
__global__ __launch_bounds__(256) void muon_copy_kernel(MuonBuffers b, float mul, uint16_t *out, MuonView ov)
{
    const int e = blockIdx.z, i = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
    if (i >= ov.m || j >= ov.n)
        return;
    const int64_t at = (int64_t)e * b.mp * b.np + (int64_t)i * b.np + j;
    out[e * ov.se + i * ov.si + j * ov.sj] = __builtin_bit_cast(uint16_t, (__bf16)(join_half(b.xh[at], b.xl[at]) * mul));
}

}  // namespace mxq
