// Newton-Schulz orthogonalisation of weight updates (the Muon optimiser's
// step on expert weights), on the matrix cores.
//
// Per matrix, X of m <= n (a tall matrix is taken transposed):
//   X = G / (|G|_F + eps);  `steps` times:  A = X X^T,  B = bA + cA^2,
//   X = aX + BX;            out = scale * X.
//
// Three products per step.  A and A^2 are symmetric: only the tiles on and
// below the diagonal are computed, each stored a second time mirrored.
// The long sums of a long matrix's A are split over workgroups and joined.
//
// Numerics.  The products run on f16 MFMA with fp32 accumulators.  f16 keeps
// 11 bits; X, A and B have magnitudes known from the iteration (|X|_2 <= 1.3
// for the usual coefficients), so fixed powers of two (kScaleX, kScaleA,
// kScaleB) keep them far from f16's ends.  Rounding the operands alone would
// cost 1.4e-3 to 3e-3 of the result (relative 2-norm, simulated), more than
// the final bf16 rounding (1.65e-3).  Two exact rearrangements bring it to
// 2e-4 to 7e-4 for ordinary gradients without another product:
//   - X is carried in two parts, f16 and the difference in e4m3 (about 15
//     bits; 22 bits of f16 + f16 measured no better and cost a byte per element
//     each way), and a X + diag(B) X is added in fp32 from both parts; only the
//     product with the rest of B sees the f16 part alone;
//   - the diagonals d of A and of B, which are the large entries when the
//     singular values are near one another, never enter an f16 operand: with
//     A = diag(d) + O,  A^2 = O O + d_i O_ij + O_ij d_j + diag(d^2), and the
//     last three terms are fp32 in the epilogue (O there from two parts).
// Where O is large instead (rows that repeat, gradients of few tokens), f16's
// roundings of O and B come back, without those of the diagonals that would
// meet them: with the output's rounding 2e-3 to 4e-3, for one token 4e-3 to
// 1.3e-2.  The same steps on bf16 operands are 2e-2 off for ordinary gradients
// and of no use for those of one token (1.2).
//
// Layout.  X is row-major.  X X^T and O O sum along rows; B X sums along X's
// columns and reads its operand through the transposing LDS read, so X is
// stored once (two high parts in turn, since B X reads whole columns of one
// while the other is written).  Buffers are padded with zeros to whole tiles,
// so the products need no bounds checks: padding stays zero through the steps.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "moe_rows_kernels.hpp"
#include "mxq_device.hpp"
#include "tile_ops.hpp"
#include "wave_ops.hpp"

namespace mxq {

constexpr float kScaleX = 8192.0f;   // |x| <= 1.3: up to 10650; room to 8
constexpr float kScaleA = 2048.0f;   // |o| <= 1.7; room to 32
constexpr float kScaleB = 2048.0f;   // |b| <= 3; room to 32
constexpr float kLow = 64.0f;        // low parts are stored times this: half an f16 ulp of 10650 is 4, e4m3 ends at 448
constexpr int kBand = 8;              // row tiles of a band (order of the tiles)
constexpr int kNormParts = 512;      // at most this many partial sums of a matrix's squared norm
constexpr int kNormThreads = 512, kNormLoads = 4;

// Buffers of one call; matrix e's parts are `e` strides further.
struct MuonBuffers {
    _Float16 *xh[2];        // [mp][np] X, this step's and the next
    uint8_t *xl;            // [mp][np] its low part
    _Float16 *oh, *bo;      // [mp][mp] off-diagonal A and B
    uint8_t *ol;            // [mp][mp] A's low part
    float *d, *db;          // [mp] diagonals of A and B
    double *part;           // [kNormParts] partial sums of squares
    int mp, np;             // padded extents
    __device__ __forceinline__ float *sums(int cur) const { return reinterpret_cast<float *>(xh[cur ^ 1]); }
    int parts;              // partial sums in use
    int splits;             // parts of X X^T's sum, 1: none
};

struct MuonView {           // x(i, j) = p[e * se + i * si + j * sj], i < m, j < n
    int64_t se, si, sj;
    int m, n;
};

// eight values as f16 and the e4m3 codes of what f16 left of them
__device__ __forceinline__ void split8(const float (&v)[8], half8 &hi, uint2 &lo)
{
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        hi[k] = (_Float16)v[k];
        r[k] = (v[k] - (float)hi[k]) * kLow;
    }
    lo.x = cvt4(r[0], r[1], r[2], r[3]);
    lo.y = cvt4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ void join8(const half8 &hi, const uint2 &lo, float (&v)[8])
{
    typedef float float2v __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const float2v a = __builtin_amdgcn_cvt_pk_f32_fp8((int)(q ? lo.y : lo.x), false);
        const float2v b = __builtin_amdgcn_cvt_pk_f32_fp8((int)(q ? lo.y : lo.x), true);
        v[4 * q] = fmaf(a[0], 1.0f / kLow, (float)hi[4 * q]);
        v[4 * q + 1] = fmaf(a[1], 1.0f / kLow, (float)hi[4 * q + 1]);
        v[4 * q + 2] = fmaf(b[0], 1.0f / kLow, (float)hi[4 * q + 2]);
        v[4 * q + 3] = fmaf(b[1], 1.0f / kLow, (float)hi[4 * q + 3]);
    }
}

// ---------------------------------------------------------------- norm, load

// Squares in fp64: no value of a finite bf16 or fp32 matrix over- or
// underflows, and the rate does not matter beside the reads.  The matrix is
// read along its unit-stride dim, 16 bytes per lane, as `outer` rows of
// `inner` elements (one row when it is contiguous), by up to kNormParts
// workgroups: one matrix alone needs two of 8 waves per CU with four loads
// each on their way.  One 8192 x 5120 bf16 21.5 us (3.9 TB/s; 49 us with one
// workgroup of 4 waves per CU), 32 of 2048 x 768 25 us.
template <typename T>
__global__ __launch_bounds__(kNormThreads) void muon_norm_kernel(const T *__restrict__ g, int64_t se, int64_t inner,
                                                                 int64_t outer, int64_t so, double *part)
{
    constexpr int N = Piece<T>::N;
    __shared__ double sums[kNormThreads / 64];
    const int e = blockIdx.y;
    const T *p = g + e * se;
    double s = 0.0;
    const int64_t span = kNormThreads * N * kNormLoads, chunks = (inner + span - 1) / span;
    for (int64_t item = blockIdx.x; item < outer * chunks; item += gridDim.x) {
        const int64_t o = item / chunks, i0 = (item - o * chunks) * span + threadIdx.x * N;
        const T *row = p + o * so;
#pragma unroll
        for (int u = 0; u < kNormLoads; ++u) {
            const int64_t i = i0 + u * kNormThreads * N;
            if (i + N <= inner) {
                const Piece<T> v = ld_piece<T>(row + i);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    s = fma((double)v.get(k), (double)v.get(k), s);
            } else {
                for (int64_t k = i; k < inner; ++k) {
                    const double x = (double)Piece<T>::to_f32(row[k]);
                    s = fma(x, x, s);
                }
            }
        }
    }
    s = block_sum<kNormThreads>(sums, s);
    if (threadIdx.x == 0)
        part[(int64_t)e * kNormParts + blockIdx.x] = s;
}

// X = G / (norm + eps) into the padded buffers, 64 x 64 elements per
// workgroup.  A lane takes 8 elements along G's unit-stride dim and passes
// them through LDS to lanes that hold 8 along X's rows.  One 8192 x 5120 bf16
// 35 us for 210 MB (6.0 TB/s), bound by memory.
template <typename T>
__global__ __launch_bounds__(256) void muon_load_kernel(const T *__restrict__ g, MuonView v, MuonBuffers b, float eps)
{
    __shared__ float tile[64][65];
    __shared__ double sums[4];
    const int tid = threadIdx.x;
    const int e = blockIdx.z, i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    double square = 0.0;
    for (int i = tid; i < b.parts; i += 256)
        square += b.part[(int64_t)e * kNormParts + i];
    square = block_sum<256>(sums, square);
    // in fp64: the reciprocal of a tiny norm overflows fp32.  A matrix of zeros
    // stays zeros with eps = 0 too.
    const double norm = sqrt(square) + (double)eps, mul = norm == 0.0 ? 0.0 : (double)kScaleX / norm;
    const T *p = g + e * v.se;
    const bool inner_j = v.sj == 1;
    const int n_in = inner_j ? v.n - j0 : v.m - i0, n_out = inner_j ? v.m - i0 : v.n - j0;
    const int64_t so = inner_j ? v.si : v.sj;
    p += inner_j ? (int64_t)i0 * v.si + j0 : (int64_t)j0 * v.sj + i0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int o = (tid >> 3) + 32 * h, in = (tid & 7) * 8;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = 0.0f;
        if (o < n_out) {
            const T *row = p + o * so + in;
            if (in + 8 <= n_in) {
#pragma unroll
                for (int q = 0; q < 8; q += Piece<T>::N) {
                    const Piece<T> w = ld_piece<T>(row + q);
#pragma unroll
                    for (int k = 0; k < Piece<T>::N; ++k)
                        x[q + k] = w.get(k);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (in + k < n_in)
                        x[k] = Piece<T>::to_f32(row[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float y = (float)((double)x[k] * mul);
            if (inner_j)
                tile[o][in + k] = y;
            else
                tile[in + k][o] = y;
        }
    }
    __syncthreads();
    const int64_t xo = (int64_t)e * b.mp * b.np;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = (tid >> 3) + 32 * h, j = (tid & 7) * 8;
        half8 hi;
        uint2 lo;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = tile[i][j + k];
        split8(x, hi, lo);
        const int64_t at = xo + (int64_t)(i0 + i) * b.np + j0 + j;
        *reinterpret_cast<half8 *>(b.xh[0] + at) = hi;
        *reinterpret_cast<uint2 *>(b.xl + at) = lo;
    }
}

// ---------------------------------------------------------------- products

enum MuonMode { kModeA, kModeB, kModeX, kModeOut, kModePart };

struct MuonStep {
    float a, b, c, out_scale;
    int cur;  // which xh holds X now
};

// Tile of the result, grid of waves and LDS stages of a product.
//   TM x TN  tile, WM x WN waves, BK summed elements per stage, NST stages
template <int TM_, int TN_, int WM_, int WN_, int BK_, int NST_>
struct MuonTile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, BK = BK_, NST = NST_;
    static constexpr int THREADS = WM * WN * 64;
    static constexpr int FP = TM / WM / 16, FQ = TN / WN / 16;  // 16 x 16 fragments of a wave
    static constexpr int STAGE = (TM + TN) * BK;                // f16 elements of a stage
    static constexpr int LOADS = STAGE * 2 / 16 / THREADS;      // 16-byte loads of a thread
    static constexpr int SS = TM / TN;                          // column tiles per row tile on the diagonal
    // the results pass through LDS RC rows of a wave's part at a time
    static constexpr int RC = FP * 16 < 64 ? FP * 16 : 64, WJ = FQ * 16;
    static_assert(RC * WJ * 2 * WM * WN <= NST * STAGE, "the results fit in the stages");
    static_assert(TM * BK / 8 % THREADS == 0, "a load is of P or of Q for the whole workgroup");
    static_assert(TM % TN == 0, "the diagonal blocks are whole tiles");
};

// Matrix e and tile (bi, bj) number id.  Bands of kBand row tiles, columns
// outermost in a band: the tiles that an XCD works on at a time form a block
// and share their operands in its L2.
template <typename TILE, bool SYM>
__device__ __forceinline__ void muon_tile(int id, int mp, int np, int &e, int &bi, int &bj)
{
    constexpr int SS = TILE::SS;
    const int tm = mp / TILE::TM, tn = SYM ? mp / TILE::TN : np / TILE::TN;
    const int per_matrix = SYM ? SS * (tm * (tm + 1) / 2) : tm * tn;
    e = id / per_matrix;
    int t = id % per_matrix;
    if (SYM) {
        // row tile r has the SS (r + 1) column tiles up to its diagonal block
        int r0 = 0, size = min(kBand, tm);
        for (;;) {
            const int r1 = r0 + size, band = SS * ((r1 * (r1 + 1) - r0 * (r0 + 1)) / 2);
            if (t < band)
                break;
            t -= band;
            r0 = r1;
            size = min(kBand, tm - r0);
        }
        const int full = SS * (r0 + 1) * size;
        if (t < full) {
            bj = t / size;
            bi = r0 + t % size;
        } else {
            t -= full;
            int x = 1;  // row tiles of the band that the column no longer has
            while (t >= SS * (size - x)) {
                t -= SS * (size - x);
                ++x;
            }
            bj = SS * (r0 + x) + t / (size - x);
            bi = r0 + x + t % (size - x);
        }
    } else {
        const int band = t / (kBand * tn), size = min(kBand, tm - band * kBand);
        t -= band * kBand * tn;
        bi = band * kBand + t % size;
        bj = t / size;
    }
}

// The stages of a tile's operands in LDS: loads and fragment reads.
//
// A stage holds TM rows of P, BK elements each, then Q: in the symmetric modes
// (QT false) TN rows like P's, else BK rows of TN elements.  Loads into LDS
// are linear; to spread the lanes of one LDS read over the banks, the order of
// the chunks of a row is exchanged in the addresses that are loaded.
//   16-byte chunk c of a row of P is at c ^ rswap(row).  A 16-byte LDS read
//   runs 16 lanes at a time, lanes 0-3, 12-15, 20-27 first.
//   32-byte chunk c of row k of a transposed Q is at c ^ qswap(k).
template <typename TILE, bool QT>
struct MuonStages {
    static constexpr int TM = TILE::TM, TN = TILE::TN, BK = TILE::BK, LOADS = TILE::LOADS, CH = BK / 8;
    static constexpr int PL = TM * CH / TILE::THREADS;       // loads of P, then those of Q
    static constexpr int PR = TILE::THREADS / CH;            // rows of P per load
    static constexpr int QR = QT ? TILE::THREADS / (TN / 8) : PR;
    static_assert(PR % 16 == 0 && QR % 16 == 0, "the chunk orders repeat with each load");
    // a load's address: uniform base (operand, load, stage) + this thread's offset
    const char *pbase, *qbase;
    int64_t prow, qrow, qstep;   // bytes from load to load, and of Q from stage to stage
    uint32_t poff, qoff, lds0;
    // LDS addresses of this lane's fragment reads in stage 0: by half of the
    // stage, or (transposed Q) by column fragment.  The rest of an address is
    // a constant of the instruction.
    uint32_t pread[2], qread[QT ? TILE::FQ : 2];
    int wave;

    // both depend on the row's low four bits alone
    static __device__ __forceinline__ int rswap(int r) { return (r >> 1) & 7; }
    static __device__ __forceinline__ int qswap(int k)
    {
        return TN >= 128 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    }

    // row0, col0: the wave's part of the tile
    __device__ __forceinline__ MuonStages(const _Float16 *l, const _Float16 *P, const _Float16 *Q, int K, int ldq,
                                          int w, int row0, int col0)
        : pbase(reinterpret_cast<const char *>(P)), qbase(reinterpret_cast<const char *>(Q)),
          prow((int64_t)PR * K * 2), qrow((int64_t)QR * (QT ? ldq : K) * 2), qstep(QT ? (int64_t)BK * ldq * 2 : BK * 2),
          lds0((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)l), wave(w)
    {
        const int t = threadIdx.x, r = t / CH, fr = t & 15, fk = (t & 63) >> 4;
        poff = (uint32_t)(r * K + ((t % CH) ^ rswap(r)) * 8) * 2;
        if (QT) {
            const int k = t / (TN / 8);
            qoff = (uint32_t)(k * ldq + ((t % (TN / 8)) ^ (qswap(k) << 1)) * 8) * 2;
            const int kr = 8 * fk + (fr >> 2);  // and the four rows after
#pragma unroll
            for (int j = 0; j < TILE::FQ; ++j)
                qread[j] = lds0 + (uint32_t)(TM * BK + kr * TN + ((col0 / 16 + j) ^ qswap(kr)) * 16 + (fr & 3) * 4) * 2;
        } else {
            qoff = poff;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                qread[h] = lds0 + (uint32_t)((TM + col0 + fr) * BK + ((h * 4 + fk) ^ rswap(fr)) * 8) * 2;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            pread[h] = lds0 + (uint32_t)((row0 + fr) * BK + ((h * 4 + fk) ^ rswap(fr)) * 8) * 2;
    }

    // load u of stage kt into LDS stage s
    __device__ __forceinline__ void load_one(int s, int u, int kt) const
    {
        const uint32_t dst = lds0 + (uint32_t)(s * TILE::STAGE * 2 + (u * TILE::THREADS + wave * 64) * 16);
        const char *base = u < PL ? pbase + u * prow + (int64_t)kt * (BK * 2) : qbase + (u - PL) * qrow + kt * qstep;
        load_lds16(base + (u < PL ? poff : qoff), __builtin_amdgcn_readfirstlane(dst));
    }

    __device__ __forceinline__ void load(int s, int kt) const
    {
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
            load_one(s, u, kt);
    }

    // fragments I0.. of P, and of Q, in half `ks` of a stage
    template <int I0, int N>
    __device__ __forceinline__ void read_p(int stage, int ks, half8 (&pf)[N]) const
    {
        const uint32_t a = pread[ks] + (uint32_t)(stage * TILE::STAGE * 2);
#pragma unroll
        for (int i = 0; i < N; ++i)
            pf[i] = read_lds(a + (I0 + i) * 16 * BK * 2);
    }

    __device__ __forceinline__ void read_q(int stage, int ks, half8 (&qf)[TILE::FQ]) const
    {
        const uint32_t off = (uint32_t)(stage * TILE::STAGE * 2);
#pragma unroll
        for (int j = 0; j < TILE::FQ; ++j) {
            if constexpr (!QT) {
                qf[j] = read_lds(qread[ks] + off + j * 16 * BK * 2);
            } else {
                const uint32_t a = qread[j] + off + ks * 32 * TN * 2;
                const half4 x = read_transposed(a), y = read_transposed(a + 4 * TN * 2);
                qf[j] = half8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            }
        }
    }
};

// Q is the first operand: a lane's four results lie along j
template <int I0, int N, int FQ, int FP>
__device__ __forceinline__ void multiply(const half8 (&pf)[N], const half8 (&qf)[FQ], float4v (&acc)[FP][FQ])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j)
            acc[I0 + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qf[j], pf[i], acc[I0 + i][j], 0, 0, 0);
}

// Fragments are read one half stage ahead of their MFMAs: the second half of
// stage kt beside the products of its first, then, past the stage's one
// barrier, the first half of stage kt + 1 beside the products of the second.
// At the barrier every wave has read stage kt and has stage kt + 1; the load
// of stage kt + NST overwrites stage kt.
template <typename TILE, bool QT>
__device__ __forceinline__ void run_pipeline(const MuonStages<TILE, QT> &st, int end,
                                             float4v (&acc)[TILE::FP][TILE::FQ])
{
    static_assert(TILE::BK == 64, "a stage has two halves");
    constexpr int NST = TILE::NST;
    half8 p0[TILE::FP], q0[TILE::FQ], p1[TILE::FP], q1[TILE::FQ];
    for (int s = 0; s < NST; ++s)
        if (s < end)
            st.load(s, s);
    if (end >= NST)
        wait_stage<(NST - 1) * TILE::LOADS>();
    else
        wait_stage<0>();
    st.read_q(0, 0, q0);
    st.template read_p<0>(0, 0, p0);
    int now = 0, kt = 0;
    for (; kt + 1 < end; ++kt) {
        const int next = now + 1 == NST ? 0 : now + 1;
        st.read_q(now, 1, q1);
        st.template read_p<0>(now, 1, p1);
        multiply<0>(p0, q0, acc);
        if (kt + NST <= end)
            wait_stage<(NST - 2) * TILE::LOADS>();
        else
            wait_stage<0>();
        if (kt + NST < end)
            st.load(now, kt + NST);
        st.read_q(next, 0, q0);
        st.template read_p<0>(next, 0, p0);
        multiply<0>(p1, q1, acc);
        now = next;
    }
    st.read_q(now, 1, q1);
    st.template read_p<0>(now, 1, p1);
    multiply<0>(p0, q0, acc);
    multiply<0>(p1, q1, acc);
}

// Two groups of four waves, one wave of each on every SIMD, one phase apart:
// while one group's MFMAs run the other reads its fragments.  Group 0 has the
// upper half of the tile's rows, group 1 the lower; each half's rows are taken
// in two quarters.  A stage takes four phases with a barrier after each:
//   ra  read Q and the first quarter     ma  multiply
//   rb  read the second quarter          mb  multiply
// and group 1 is in the phase before group 0's.
//
// Two stages in LDS, but a stage's parts are loaded as soon as the part that
// they overwrite has been read by both groups (a read phase ends with its
// reads returned), so every part has five phases (about 500 cycles each) to
// arrive.  Loads are issued in the read phases alone, after the LDS reads: in
// front of a phase's MFMAs they held those up.  In either group's phases of
// stage t:
//   ra(t)  quarters 1 and 3 of t + 1      (first read in rb(t + 1))
//   rb(t)  Q, quarters 0 and 2 of t + 2   (first read in ra(t + 2))
// The loads of a wave return in order: at the end of group 0's mb(t) the parts
// for ra(t + 1) have landed when only the 8 loads issued since are pending
// (2 of t + 1 and 6 of t + 2), at the end of its ma(t) those for rb(t) when
// again 8 are.  (A tile of 128 columns has two loads of Q, and 6 pending.)
template <typename TILE, bool QT>
struct MuonAlternating {
    static_assert(TILE::BK == 64 && TILE::NST == 2 && TILE::WM == 2 && TILE::WN == 4 && TILE::TM == 256,
                  "loads 0-3 are the quarters, the rest Q");
    static constexpr int H = TILE::FP / 2;
    static constexpr int FIRST = TILE::LOADS - 2;  // loads for ra
    const MuonStages<TILE, QT> &st;
    half8 p0[H], p1[H], q0[TILE::FQ], q1[TILE::FQ];

    __device__ __forceinline__ void load_a(int kt) const
    {
#pragma unroll
        for (int u = 4; u < TILE::LOADS; ++u)
            st.load_one(kt & 1, u, kt);
        st.load_one(kt & 1, 0, kt);
        st.load_one(kt & 1, 2, kt);
    }
    __device__ __forceinline__ void load_b(int kt) const
    {
        st.load_one(kt & 1, 1, kt);
        st.load_one(kt & 1, 3, kt);
    }

    __device__ __forceinline__ void read_a(int s)
    {
        st.read_q(s, 0, q0);
        st.template read_p<0>(s, 0, p0);
        st.read_q(s, 1, q1);
        st.template read_p<0>(s, 1, p1);
    }
    __device__ __forceinline__ void read_b(int s)
    {
        st.template read_p<H>(s, 0, p0);
        st.template read_p<H>(s, 1, p1);
    }
    template <int I0>
    __device__ __forceinline__ void products(float4v (&acc)[TILE::FP][TILE::FQ])
    {
        __builtin_amdgcn_s_setprio(1);
        multiply<I0>(p0, q0, acc);
        multiply<I0>(p1, q1, acc);
        __builtin_amdgcn_s_setprio(0);
    }

    // one stage; MORE: how many stages follow (0, 1, or 2 for two and more)
    template <bool LATER, int MORE>
    __device__ __forceinline__ void stage(int kt, float4v (&acc)[TILE::FP][TILE::FQ])
    {
        constexpr int kB = MORE >= 1 ? 2 + FIRST : 0;                         // pending when rb may begin
        constexpr int kNext = MORE >= 2 ? 2 + FIRST : MORE == 1 ? 2 : -1;     // when the next ra may
        const int s = kt & 1;
        read_a(s);
        if (MORE >= 1)
            load_b(kt + 1);
        phase_end<LATER ? kB : -1>();
        products<0>(acc);
        phase_end<LATER ? -1 : kB>();
        read_b(s);
        if (MORE >= 2)
            load_a(kt + 2);
        phase_end<LATER ? kNext : -1>();
        products<H>(acc);
        phase_end<LATER ? -1 : kNext>();
    }

    template <bool LATER>
    __device__ __forceinline__ void run_group(int end, float4v (&acc)[TILE::FP][TILE::FQ])
    {
        if (LATER)
            phase_end<-1>();
        int kt = 0;
        for (; kt + 2 < end; ++kt)
            stage<LATER, 2>(kt, acc);
        if (kt + 1 < end) {
            stage<LATER, 1>(kt, acc);
            ++kt;
        }
        stage<LATER, 0>(kt, acc);
        if (!LATER)
            phase_end<-1>();
    }

    __device__ __forceinline__ void run(int end, float4v (&acc)[TILE::FP][TILE::FQ])
    {
        st.load(0, 0);
        if (end > 1) {
            load_a(1);
            phase_end<FIRST>();
        } else {
            phase_end<0>();
        }
        if (st.wave >= 4)
            run_group<true>(end, acc);
        else
            run_group<false>(end, acc);
    }
};

// C[i][j] = sum_k P[i][k] Q[k][j].
//   kModeA    P = X, Q = X^T: off-diagonal A in two parts, diagonal d
//   kModeB    P = Q = O (symmetric): off-diagonal B, diagonal db
//   kModeX    P = B, Q = X: the next X in both parts
//   kModeOut  the same, to the caller's output
//   kModePart part `split` of kModeA's sum, as it is, in fp32 to where the
//             next X will be (muon_join_kernel does the rest)
template <int MODE, typename TILE>
__device__ __forceinline__ void muon_product(_Float16 *lds, const MuonBuffers &b, const MuonStep &st, uint16_t *out,
                                             const MuonView &ov, int e, int i0, int j0, bool mirror, int split)
{
    constexpr int FP = TILE::FP, FQ = TILE::FQ;
    constexpr bool SYM = MODE == kModeA || MODE == kModeB || MODE == kModePart;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / TILE::WN, wq = wave % TILE::WN;
    const int fr = threadIdx.x & 15, fk = (threadIdx.x & 63) >> 4;
    const int64_t xo = (int64_t)e * b.mp * b.np, ao = (int64_t)e * b.mp * b.mp;
    constexpr bool XX = MODE == kModeA || MODE == kModePart;
    const int K = XX ? b.np : b.mp;
    int first = 0, last = K / TILE::BK;  // stages
    if constexpr (MODE == kModePart) {
        const int all = last;
        first = split * all / b.splits;
        last = (split + 1) * all / b.splits;
    }
    const _Float16 *P = XX ? b.xh[st.cur] + xo : MODE == kModeB ? b.oh + ao : b.bo + ao;
    P += first * TILE::BK;
    const _Float16 *Q = SYM ? P + (int64_t)j0 * K : b.xh[st.cur] + xo + j0;
    MuonStages<TILE, !SYM> stages(lds, P + (int64_t)i0 * K, Q, K, b.np, wave, wp * FP * 16, wq * FQ * 16);

    // What the results are combined with, for RC rows of the wave's part.  With
    // few registers per thread it is read before the products, so that it costs
    // no wait after them.
    constexpr int RC = TILE::RC, WJ = TILE::WJ, LPR = WJ / 8, RPP = 64 / LPR, PASSES = RC / RPP;
    constexpr int CHUNKS = FP * 16 / RC;
    constexpr bool EARLY = CHUNKS == 1 && PASSES <= 2;
    const int lane = threadIdx.x & 63, pr = lane / LPR, pc = lane % LPR;
    const int wi0 = i0 + wp * FP * 16, wj0 = j0 + wq * WJ, gj = wj0 + pc * 8;
    float *d = b.d + (int64_t)e * b.mp, *db = b.db + (int64_t)e * b.mp;
    half8 oldh[2][PASSES];
    uint2 oldl[2][PASSES];
    float di[2][PASSES];
    auto load_old = [&](int ic, int set) {
        if constexpr (!XX) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int gi = wi0 + ic + p * RPP + pr;
                di[set][p] = MODE == kModeB ? d[gi] : db[gi];
                const int64_t at = MODE == kModeB ? ao + (int64_t)gi * b.mp + gj : xo + (int64_t)gi * b.np + gj;
                oldh[set][p] = *reinterpret_cast<const half8 *>((MODE == kModeB ? b.oh : b.xh[st.cur]) + at);
                oldl[set][p] = *reinterpret_cast<const uint2 *>((MODE == kModeB ? b.ol : b.xl) + at);
            }
        }
    };
    if constexpr (EARLY)
        load_old(0, 0);

    float4v acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j)
            acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (TILE::TM == 256)
        MuonAlternating<TILE, !SYM>{stages}.run(last - first, acc);
    else
        run_pipeline<TILE, !SYM>(stages, last - first, acc);

    // Results.  A lane holds row l % 16, columns 4 (l / 16) + 0..3 of each
    // fragment; through LDS (each wave in its own region, RC rows at a time)
    // it gets 8 consecutive columns of one row instead, so that everything
    // below is read and written in 16-byte pieces of whole 128-byte lines.
    // stored a second time (or only) transposed: the mirror of an off-diagonal
    // tile, and the output of a tall matrix
    const bool turned = MODE == kModePart ? false : SYM ? mirror : MODE == kModeOut && ov.si == 1 && ov.sj != 1;
    float *wide = reinterpret_cast<float *>(lds) + wave * RC * WJ;
    _Float16 *turn = reinterpret_cast<_Float16 *>(wide);
    // chunk orders of the two uses of the region: 16-byte chunks of fp32 rows,
    // 32-byte chunks of f16 rows
    auto wswap = [](int r) { return WJ == 64 ? r & 15 : (r >> 1) & 7; };
    auto tswap = [](int r) { return WJ == 64 ? ((r >> 1) & 1) | ((r >> 3) & 1) << 1 : (r >> 3) & 1; };
    if constexpr (!EARLY)
        load_old(0, 0);
    float dj[8];
    if constexpr (MODE == kModeB)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            dj[k] = d[gj + k];
    wait_stage<0>();  // every wave is done with the stages
#pragma unroll
    for (int ch = 0; ch < CHUNKS; ++ch) {
        const int ic = ch * RC, set = ch & 1;
#pragma unroll
        for (int i = 0; i < RC / 16; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j)
                *reinterpret_cast<float4v *>(wide + (i * 16 + fr) * WJ + ((4 * j + fk) ^ wswap(i * 16 + fr)) * 4) =
                    acc[ic / 16 + i][j];
        if (ch + 1 < CHUNKS)
            load_old(ic + RC, set ^ 1);
        __builtin_amdgcn_wave_barrier();
        half8 h8[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + pr, gi = wi0 + ic + r;
            float v[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4v x = *reinterpret_cast<const float4v *>(wide + r * WJ + ((2 * pc + q) ^ wswap(r)) * 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[4 * q + k] = x[k];
            }
            uint2 low;
            if constexpr (MODE == kModePart) {
                float *o = b.sums(st.cur) + (int64_t)split * ov.se + ao + (int64_t)gi * b.mp + gj;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    reinterpret_cast<float4v *>(o)[q] = float4v{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            } else if constexpr (MODE == kModeA) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[k] *= 1.0f / (kScaleX * kScaleX);
                    const bool diag = gi == gj + k;
                    if (diag)
                        d[gi] = v[k];
                    v[k] = diag ? 0.0f : v[k] * kScaleA;
                }
                split8(v, h8[p], low);
                const int64_t at = ao + (int64_t)gi * b.mp + gj;
                *reinterpret_cast<half8 *>(b.oh + at) = h8[p];
                *reinterpret_cast<uint2 *>(b.ol + at) = low;
            } else if constexpr (MODE == kModeB) {
                const float dg = di[set][p];
                float o[8];
                join8(oldh[set][p], oldl[set][p], o);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float oo = v[k] * (1.0f / (kScaleA * kScaleA)), ok = o[k] * (1.0f / kScaleA);
                    const bool diag = gi == gj + k;
                    const float aij = diag ? dg : ok;
                    const float a2 = oo + (diag ? dg * dg : (dg + dj[k]) * ok);
                    const float x = st.b * aij + st.c * a2;
                    if (diag)
                        db[gi] = x;
                    h8[p][k] = (_Float16)(diag ? 0.0f : x * kScaleB);
                }
                *reinterpret_cast<half8 *>(b.bo + ao + (int64_t)gi * b.mp + gj) = h8[p];
            } else {
                const float own = st.a + di[set][p];
                float x[8];
                join8(oldh[set][p], oldl[set][p], x);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = fmaf(own, x[k], v[k] * (1.0f / kScaleB));
                if constexpr (MODE == kModeX) {
                    split8(x, h8[p], low);
                    const int64_t at = xo + (int64_t)gi * b.np + gj;
                    *reinterpret_cast<half8 *>(b.xh[st.cur ^ 1] + at) = h8[p];
                    *reinterpret_cast<uint2 *>(b.xl + at) = low;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        h8[p][k] = __builtin_bit_cast(_Float16, (__bf16)(x[k] * st.out_scale));
                    if (!turned && gi < ov.m) {
                        typedef _Float16 Out8 __attribute__((ext_vector_type(8), aligned(2)));
                        _Float16 *o = reinterpret_cast<_Float16 *>(out) + e * ov.se + (int64_t)gi * ov.si;
                        if (ov.sj == 1 && gj + 8 <= ov.n) {
                            *reinterpret_cast<Out8 *>(o + gj) = h8[p];
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (gj + k < ov.n)
                                    o[(int64_t)(gj + k) * ov.sj] = h8[p][k];
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if (MODE == kModeX || MODE == kModePart || !turned)
            continue;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + pr;
            *reinterpret_cast<half8 *>(turn + r * WJ + (((pc >> 1) ^ tswap(r)) * 2 + (pc & 1)) * 8) = h8[p];
        }
        __builtin_amdgcn_wave_barrier();
        // lane l reads column l % 16 of rows 8 (l / 16) + 0..7 of a block of 32
        const uint32_t turn0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)turn;
#pragma unroll
        for (int i = 0; i < RC; i += 32)
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const int r = i + 8 * fk + (fr >> 2), c = (fr & 3) * 4;
                const half4 a = read_transposed(turn0 + (r * WJ + (j ^ tswap(r)) * 16 + c) * 2);
                const half4 h = read_transposed(turn0 + ((r + 4) * WJ + (j ^ tswap(r + 4)) * 16 + c) * 2);
                const half8 w = {a[0], a[1], a[2], a[3], h[0], h[1], h[2], h[3]};
                const int gi = wi0 + ic + i + 8 * fk, gj = wj0 + 16 * j + fr;  // of this lane's column
                if constexpr (SYM) {
                    _Float16 *o = (MODE == kModeA ? b.oh : b.bo) + ao + (int64_t)gj * b.mp + gi;
                    *reinterpret_cast<half8 *>(o) = w;
                } else if (gj < ov.n) {
                    typedef _Float16 Out8 __attribute__((ext_vector_type(8), aligned(2)));
                    _Float16 *o = reinterpret_cast<_Float16 *>(out) + e * ov.se + (int64_t)gj * ov.sj + gi;
                    if (gi + 8 <= ov.m) {
                        *reinterpret_cast<Out8 *>(o) = w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (gi + k < ov.m)
                                o[k] = w[k];
                    }
                }
            }
        __builtin_amdgcn_wave_barrier();
    }
}

// `whole` workgroups take a tile each; of the tiles after those, two
// workgroups take the column halves.
//
// One 8192 x 5120, per launch: X X^T 178 us (1.27 PFLOP/s of the half that is
// computed; MFMA busy 82%), A^2 121 us (1.16), B X 362 us (1.19, MFMA busy
// 61%): bound by the matrix units at the clock they sustain (a library
// product of 16384 x 16384 x 8192 f16 reaches 1.33 PFLOP/s here).  32 of
// 2048 x 768: 60, 37 and 116 us: the 192 tiles of the first two leave a
// quarter of the CUs idle, and X X^T and B X pass 450 MB and more through the
// Infinity Cache around 12 to 32 stages per tile.  One 512 x 512: 6 to 7.6
// us, of which 2.3 are the launch and the rest the latency of 8 dependent
// stages and of operands that other XCDs have just written.
template <int MODE, typename TILE, typename HALF>
__global__ __launch_bounds__(TILE::THREADS, 2) void muon_product_kernel(MuonBuffers b, MuonStep st, uint16_t *out,
                                                                     MuonView ov, int whole)
{
    constexpr bool SYM = MODE == kModeA || MODE == kModeB || MODE == kModePart;
    __shared__ __attribute__((aligned(16))) _Float16 lds[TILE::NST * TILE::STAGE];
    int e, bi, bj;
    if constexpr (MODE == kModePart) {
        const int id = xcd_run(blockIdx.x, gridDim.x);
        muon_tile<TILE, true>(id % whole, b.mp, b.np, e, bi, bj);
        muon_product<MODE, TILE>(lds, b, st, out, ov, e, bi * TILE::TM, bj * TILE::TN, false, id / whole);
    } else if ((int)blockIdx.x < whole) {
        muon_tile<TILE, SYM>(xcd_run(blockIdx.x, whole), b.mp, b.np, e, bi, bj);
        muon_product<MODE, TILE>(lds, b, st, out, ov, e, bi * TILE::TM, bj * TILE::TN, bj < bi * TILE::SS, 0);
    } else if constexpr (!std::is_same<TILE, HALF>::value) {
        const int id = xcd_run(blockIdx.x - whole, gridDim.x - whole);
        muon_tile<TILE, SYM>(whole + (id >> 1), b.mp, b.np, e, bi, bj);
        muon_product<MODE, HALF>(lds, b, st, out, ov, e, bi * TILE::TM, bj * TILE::TN + (id & 1) * HALF::TN,
                                 bj < bi * TILE::SS, 0);
    }
}

// The parts of X X^T's sum, in order, to A: a 64 x 64 tile on or below the
// diagonal per workgroup, 16 columns of a row per thread.  `whole`: elements
// from part to part.  Bound by latency (a launch and the parts' reads).
__global__ __launch_bounds__(256) void muon_join_kernel(MuonBuffers b, MuonStep st, int64_t whole)
{
    __shared__ __attribute__((aligned(16))) _Float16 tile[64][72];
    __shared__ __attribute__((aligned(16))) uint8_t tail[64][72];
    int bi = 0, t = blockIdx.x;
    while (t > bi)
        t -= ++bi;
    const int bj = t, r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
    const int64_t ao = (int64_t)blockIdx.y * b.mp * b.mp;
    const int gi = bi * 64 + r, gj = bj * 64 + c;
    const int64_t at = ao + (int64_t)gi * b.mp + gj;
    const float *p = b.sums(st.cur) + at;
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
        v[k] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < b.splits; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4v x = reinterpret_cast<const float4v *>(p + i * whole)[q];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[4 * q + k] += x[k];
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = v[8 * h + k] * (1.0f / (kScaleX * kScaleX));
            const bool diag = gi == gj + 8 * h + k;
            if (diag)
                b.d[(int64_t)blockIdx.y * b.mp + gi] = x;
            w[k] = diag ? 0.0f : x * kScaleA;
        }
        half8 hi;
        uint2 low;
        split8(w, hi, low);
        *reinterpret_cast<half8 *>(b.oh + at + 8 * h) = hi;
        *reinterpret_cast<uint2 *>(b.ol + at + 8 * h) = low;
        *reinterpret_cast<half8 *>(&tile[r][c + 8 * h]) = hi;
        *reinterpret_cast<uint2 *>(&tail[r][c + 8 * h]) = low;
    }
    if (bi == bj)
        return;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        half8 w;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = tile[c + 8 * h + k][r];
        const int64_t to = ao + (int64_t)(bj * 64 + r) * b.mp + bi * 64 + c + 8 * h;
        *reinterpret_cast<half8 *>(b.oh + to) = w;
        // the next product reads the low part of whole tiles on the diagonal
        uint2 low = {0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            low.x |= (uint32_t)tail[c + 8 * h + k][r] << (8 * k);
            low.y |= (uint32_t)tail[c + 8 * h + 4 + k][r] << (8 * k);
        }
        *reinterpret_cast<uint2 *>(b.ol + to) = low;
    }
}

// With no steps the result is scale * X itself.
__global__ __launch_bounds__(256) void muon_copy_kernel(MuonBuffers b, float mul, uint16_t *out, MuonView ov)
{
    const int e = blockIdx.z, i = blockIdx.x, j = blockIdx.y * 256 + threadIdx.x;
    if (i >= ov.m || j >= ov.n)
        return;
    const int64_t at = (int64_t)e * b.mp * b.np + (int64_t)i * b.np + j;
    const float low = __builtin_amdgcn_cvt_f32_fp8((int)b.xl[at], 0);
    out[e * ov.se + i * ov.si + j * ov.sj] =
        __builtin_bit_cast(uint16_t, (__bf16)(fmaf(low, 1.0f / kLow, (float)b.xh[0][at]) * mul));
}

}  // namespace mxq
