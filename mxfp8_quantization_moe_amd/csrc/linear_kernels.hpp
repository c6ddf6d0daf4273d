// Products of token groups with their experts' weights, on the matrix cores.
//
//   forward   z_r = W_e x_r + b_e           for the rows r of group e
//             y_r = act(z_r) + resid_r      or, gated, act(gate) * value with
//                                           the halves of z_r
//   grad x    dx_r = dz_r W_e
//   grad W    dW_e = sum over the group's rows of dz_r x_r^T
// The forward product also takes MXFP8 operands (e4m3 values, an e8m0 scale
// for 32 of them).
//
// One form carries all of them: C[i][j] = sum_k P(i, k) Q(j, k), tiles of C per
// workgroup, 128 bytes of k per row and stage.  An operand whose rows run along
// k ("rows") is read from LDS 16 bytes per lane; one whose rows run along i or
// j ("turned") through the transposing LDS read, so nothing is transposed in
// memory.  Operands go from global memory straight into LDS through buffer
// descriptors whose range ends with the group's (or the matrix's) last element:
// what lies past it arrives as zeros, in both operands, so odd lengths need no
// branch and no memory past an operand is read.
//
// Group ends stay on the device.  A workgroup finds its tile by a scan over
// the groups' tile counts in each of its waves; the grid is an upper bound and
// what is over ends at once.  Rows behind the last group are a last group whose
// results are zeros.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_ops.hpp"
#include "moe_rows_kernels.hpp"
#include "mxq_device.hpp"
#include "tile_ops.hpp"
#include "wave_ops.hpp"

namespace mxq {

enum LinearMode { kForward, kGradX, kGradW };
// Operands and results of a call; leading strides in bytes for what is read
// into LDS, else in elements.
struct LinearArgs {
    const char *p, *q;            // see the modes
    int64_t ldp, ldq, qe;         // qe: from expert to expert
    const uint8_t *sp, *sq;       // e8m0 scales (MXFP8), rows of whole words
    int64_t ldsp, ldsq, sqe;
    const int32_t *offs;          // NULL: one group of all rows
    int experts, rows;
    int width, wide;              // inner extents: of x, and of z
    int n;                        // columns of the result (wide, half of it if gated, or width)
    const void *bias;             // (experts, wide), fp32 or bf16
    int64_t sb;
    int bias_f32, act;
    const uint16_t *resid;
    int64_t sr;
    uint16_t *out, *pre;          // pre: z, forward only
    int64_t so, spre, oe;         // oe: grad W, from expert to expert
};

// ---------------------------------------------------------------- groups

// Rows [start, start + len) of group g; group `experts` is what lies behind.
__device__ __forceinline__ void group_rows(const int32_t *__restrict__ offs, int experts, int rows, int g, int &start,
                                           int &len)
{
    const int s = offs && g > 0 ? min(max(offs[min(g, experts) - 1], 0), rows) : 0;
    const int e = offs && g < experts ? min(max(offs[g], 0), rows) : rows;
    start = s;
    len = g <= experts && (offs || g < experts) ? max(e - s, 0) : 0;
}

// Tiles of TM rows of all groups, the rows behind the last one included.
template <int TM>
__device__ __forceinline__ int count_row_tiles(const LinearArgs &a)
{
    if (!a.offs)
        return (a.rows + TM - 1) / TM;
    int n = 0, start, len;
    for (int g = threadIdx.x & 63; g <= a.experts; g += 64) {
        group_rows(a.offs, a.experts, a.rows, g, start, len);
        n += (len + TM - 1) / TM;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        n += __shfl_xor(n, m, 64);
    return uniform(n);
}

// Row tile `t`: its group, first row, and rows of the group from there on.
template <int TM>
__device__ __forceinline__ void find_row_tile(const LinearArgs &a, int t, int &e, int &row0, int &left)
{
    if (!a.offs) {
        e = 0;
        row0 = t * TM;
        left = a.rows - row0;
        return;
    }
    for (int g0 = 0;; g0 += 64) {
        int start, len;
        group_rows(a.offs, a.experts, a.rows, g0 + (threadIdx.x & 63), start, len);
        const int tiles = (len + TM - 1) / TM, upto = wave_scan(tiles);
        const uint64_t past = __ballot(upto > t);
        if (past || g0 + 64 > a.experts) {
            const int lane = past ? __builtin_ctzll(past) : 63;
            const int skip = (t - (__builtin_amdgcn_readlane(upto, lane) - __builtin_amdgcn_readlane(tiles, lane))) * TM;
            e = g0 + lane;
            row0 = __builtin_amdgcn_readlane(start, lane) + skip;
            left = __builtin_amdgcn_readlane(len, lane) - skip;
            return;
        }
        t -= __builtin_amdgcn_readlane(upto, 63);
    }
}

// Workgroups go to the 8 XCDs in turn.  Number `block` of the grid in an order
// that gives an XCD runs of up to 32 tiles, a CU each, from all over the
// result: the runs share operands in its L2, and groups of any length load the
// XCDs alike.  The grid is a multiple of 256.
__device__ __forceinline__ int spread(int block, int total)
{
    const int run = max(1, min(32, (total + 7) >> 3)), s = block >> 3;
    return ((s / run) * 8 + (block & 7)) * run + s % run;
}

constexpr int kLinearBand = 8;  // row tiles of a band: a run of 32 is 8 x 4 tiles

__device__ __forceinline__ void band_tile(int t, int tm, int tn, int &bi, int &bj)
{
    const int band = t / (kLinearBand * tn), size = min(kLinearBand, tm - band * kLinearBand);
    t -= band * kLinearBand * tn;
    bi = band * kLinearBand + t % size;
    bj = t / size;
}

// ---------------------------------------------------------------- operands

// TM x TN tile, WM x WN waves, NST stages of 128 bytes of k in LDS
template <int TM_, int TN_, int WM_, int WN_, int NST_>
struct LinearTile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NST = NST_;
    static constexpr int THREADS = WM * WN * 64;
    static constexpr int FP = TM / WM / 16, FQ = TN / WN / 16;  // 16 x 16 fragments of a wave
    static constexpr int STAGE = (TM + TN) * 128;               // bytes
    // the results pass through LDS RC rows of a wave's part at a time
    static constexpr int RC = FP * 16 < 64 ? FP * 16 : 64, WJ = FQ * 16;
    static_assert(RC * WJ * 4 * WM * WN <= NST * STAGE, "the results fit in the stages");
    static_assert(THREADS >= TM + TN, "one load of scales per thread and stage");
};

// k of a stage
constexpr int kRowBytes = 128;

// One operand of a tile: EXT rows of 128 bytes, or turned 64 rows of EXT
// elements of bf16, THREADS threads.
//
// Loads into LDS are linear; to spread the lanes of one LDS read over the
// banks, the order of the chunks of a row is exchanged in the addresses that
// are loaded: 16-byte chunk c of row r is at c ^ rswap(r), 32-byte chunk c of
// a turned row k at c ^ tswap(k).
template <int EXT, int THREADS, bool TURNED>
struct Panel {
    static constexpr int CH = TURNED ? EXT / 8 : 8;       // 16-byte chunks of a row
    static constexpr int RPL = THREADS / CH;              // rows per load
    static constexpr int LOADS = EXT * 8 / THREADS;
    static_assert(RPL % 16 == 0, "the chunk orders repeat with each load");
    const char *base;
    int64_t step;                 // bytes from stage to stage
    int64_t ld;
    uint32_t off[LOADS];          // of this thread's chunks
    uint32_t range;               // bytes from base on (rows), of a row (turned)
    int rows;                     // turned: rows from base on
    int chunk;                    // this thread's chunk of k

    static __device__ __forceinline__ int rswap(int r) { return (r >> 1) & 7; }
    static __device__ __forceinline__ int tswap(int k)
    {
        return EXT >= 128 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    }

    // row(r): the operand's row that tile row r holds, relative to base, or -1
    template <typename Row>
    __device__ __forceinline__ void set_rows(const char *b, int64_t stride, uint32_t bytes, Row &&row)
    {
        base = b;
        ld = stride;
        step = kRowBytes;
        range = bytes;
        const int r = threadIdx.x / CH;
        chunk = (threadIdx.x % CH) ^ rswap(r);
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int at = row(r + u * RPL);
            off[u] = at < 0 ? 0x80000000u : (uint32_t)(at * (uint32_t)stride + chunk * 16);
        }
    }

    // `n` rows of `bytes` bytes from b on
    __device__ __forceinline__ void set_turned(const char *b, int64_t stride, uint32_t bytes, int n)
    {
        base = b;
        ld = stride;
        step = 64 * stride;
        range = bytes;
        rows = n;
        chunk = 0;
        const int k = threadIdx.x / CH;
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
            off[u] = (uint32_t)((k + u * RPL) * (uint32_t)stride + ((threadIdx.x % CH) ^ (tswap(k) << 1)) * 16);
    }

    // load u of stage kt to lds + 16 * thread; `live`: chunks of k of the stage
    __device__ __forceinline__ void load(int u, int kt, int live, uint32_t lds) const
    {
        const uint32_t bytes = TURNED ? (uint32_t)((min(rows - kt * 64, 64) - 1) * ld) + range
                                      : range - (uint32_t)(kt * kRowBytes);
        __amdgpu_buffer_rsrc_t rs = buffer_rsrc(base + kt * step, bytes);
        uint32_t o = off[u];
        if (!TURNED && live < 8)
            o = chunk < live ? o : 0x80000000u;
        const uint32_t dst = lds + (uint32_t)(u * THREADS + (threadIdx.x & ~63)) * 16;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void *)(uintptr_t)uniform((int)dst), 16, (int)o, 0, 0, 0);
    }

    // LDS addresses of this lane's fragment reads: N fragments from tile row
    // (or column) `first` on
    template <int N>
    struct Reads {
        uint32_t a[TURNED ? N : 2];
        __device__ __forceinline__ Reads(uint32_t lds, int first)
        {
            const int fr = threadIdx.x & 15, fk = (threadIdx.x & 63) >> 4;
            if constexpr (TURNED) {
                const int kr = 8 * fk + (fr >> 2);  // and the four rows after
#pragma unroll
                for (int i = 0; i < N; ++i)
                    a[i] = lds + (uint32_t)(kr * EXT + ((first / 16 + i) ^ tswap(kr)) * 16 + (fr & 3) * 4) * 2;
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    a[h] = lds + (uint32_t)((first + fr) * 128 + ((h * 4 + fk) ^ rswap(fr)) * 16);
            }
        }
        // fragments I0.. of half h of the stage `at` bytes further
        template <int I0, int M>
        __device__ __forceinline__ void read(uint32_t at, int h, half8 (&f)[M]) const
        {
#pragma unroll
            for (int i = 0; i < M; ++i) {
                if constexpr (TURNED) {
                    const uint32_t b = a[I0 + i] + at + h * 32 * EXT * 2;
                    const half4 x = read_transposed(b), y = read_transposed(b + 4 * EXT * 2);
                    f[i] = half8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                } else {
                    f[i] = read_lds(a[h] + at + (I0 + i) * 16 * 128);
                }
            }
        }
    };
};

typedef int int8v __attribute__((ext_vector_type(8)));
// acc += P Q over a stage, fragments I0.. of P.  Q is the first operand: a
// lane's four results lie along j.  The scaled product takes both halves of a
// stage at once (128 values of k): lane 16 b + i holds bytes 16 b and 64 + 16 b
// of row i and supplies the scale of its 32-value block b.
template <bool MX, int I0, int N, int FP, int FQ>
__device__ __forceinline__ void multiply_stage(const half8 (&p0)[N], const half8 (&p1)[N], const half8 (&q0)[FQ],
                                               const half8 (&q1)[FQ], const int (&sp)[N], const int (&sq)[FQ],
                                               float4v (&acc)[FP][FQ])
{
    if constexpr (MX) {
        struct Pair {
            half8 a, b;
        };
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j)
                acc[I0 + i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    __builtin_bit_cast(int8v, Pair{q0[j], q1[j]}), __builtin_bit_cast(int8v, Pair{p0[i], p1[i]}),
                    acc[I0 + i][j], 0, 0, 0, sq[j], 0, sp[i]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    acc[I0 + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, h ? q1[j] : q0[j]), __builtin_bit_cast(bf16x8, h ? p1[i] : p0[i]),
                        acc[I0 + i][j], 0, 0, 0);
    }
}

// Both operands of a tile and, for MXFP8, the scales of their rows: a word of
// four blocks per row and stage.
template <typename TILE, bool PT, bool QT, bool MX>
struct LinearStages {
    typedef Panel<TILE::TM, TILE::THREADS, PT> PanelP;
    typedef Panel<TILE::TN, TILE::THREADS, QT> PanelQ;
    static constexpr int LP = PanelP::LOADS, LQ = PanelQ::LOADS, LOADS = LP + LQ + (MX ? 1 : 0);
    static constexpr int BYTES = TILE::STAGE + (MX ? TILE::THREADS * 4 : 0);
    PanelP p;
    PanelQ q;
    const uint8_t *scales;        // this thread's row
    int stages, live;             // live: chunks of k in the last stage
    uint32_t lds0;

    __device__ __forceinline__ void load_one(int s, int u, int kt) const
    {
        const uint32_t at = lds0 + s * BYTES;
        const int n = kt + 1 < stages ? 8 : live;
        if (u < LP) {
            p.load(u, kt, n, at);
        } else if (u < LP + LQ) {
            q.load(u - LP, kt, n, at + TILE::TM * 128);
        } else {
            const uint32_t dst = at + TILE::STAGE + (threadIdx.x & ~63) * 4;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(scales + kt * 4),
                                             (__attribute__((address_space(3))) void *)(uintptr_t)uniform((int)dst), 4, 0, 0);
        }
    }
    __device__ __forceinline__ void load(int s, int kt) const
    {
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
            load_one(s, u, kt);
    }

    // scales of N fragments from tile row `first` on (of Q: TM further), each
    // lane its block's; blocks past k (whose values are zeros) count as 2^-127
    template <int N>
    __device__ __forceinline__ void read_scales(int s, int kt, int first, int (&v)[N]) const
    {
        if constexpr (MX) {
            const int fr = threadIdx.x & 15, fk = (threadIdx.x & 63) >> 4;
            const uint32_t a = lds0 + s * BYTES + TILE::STAGE + (uint32_t)(first + fr) * 4;
            const bool there = kt + 1 < stages || 2 * fk < live;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t w = *(__attribute__((address_space(3))) const uint32_t *)(uintptr_t)(a + i * 64);
                v[i] = there ? (int)((w >> (8 * fk)) & 0xffu) : 0;
            }
        }
    }
};

// Fragments are read one stage ahead of their MFMAs.  At a stage's one barrier
// every wave has read stage kt and has stage kt + 1; the load of stage kt + NST
// overwrites stage kt.
template <typename TILE, bool PT, bool QT, bool MX>
__device__ __forceinline__ void linear_pipeline(const LinearStages<TILE, PT, QT, MX> &st, int row0, int col0,
                                                float4v (&acc)[TILE::FP][TILE::FQ])
{
    typedef LinearStages<TILE, PT, QT, MX> S;
    constexpr int NST = TILE::NST, FP = TILE::FP, FQ = TILE::FQ;
    const typename S::PanelP::template Reads<FP> rp(st.lds0, row0);
    const typename S::PanelQ::template Reads<FQ> rq(st.lds0 + TILE::TM * 128, col0);
    struct Frags {
        half8 p0[FP], p1[FP], q0[FQ], q1[FQ];
        int sp[FP], sq[FQ];
    } f[2];
    auto read = [&](int s, int kt, Frags &x) {
        const uint32_t at = s * S::BYTES;
        rq.template read<0>(at, 0, x.q0);
        rp.template read<0>(at, 0, x.p0);
        rq.template read<0>(at, 1, x.q1);
        rp.template read<0>(at, 1, x.p1);
        st.read_scales(s, kt, row0, x.sp);
        st.read_scales(s, kt, TILE::TM + col0, x.sq);
    };
    const int end = st.stages;
    for (int s = 0; s < NST; ++s)
        if (s < end)
            st.load(s, s);
    if (end >= NST)
        wait_stage<(NST - 1) * S::LOADS>();
    else
        wait_stage<0>();
    read(0, 0, f[0]);
    int now = 0, kt = 0;
    auto step = [&](Frags &x, Frags &y) {
        const int next = now + 1 == NST ? 0 : now + 1;
        if (kt + 1 < end) {
            if (kt + NST <= end)
                wait_stage<(NST - 2) * S::LOADS>();
            else
                wait_stage<0>();
            if (kt + NST < end)
                st.load(now, kt + NST);
            read(next, kt + 1, y);
        }
        multiply_stage<MX, 0>(x.p0, x.p1, x.q0, x.q1, x.sp, x.sq, acc);
        now = next;
        ++kt;
    };
    while (kt + 1 < end) {
        step(f[0], f[1]);
        step(f[1], f[0]);
    }
    if (kt < end)
        step(f[0], f[1]);
}

// ---------------------------------------------------------------- epilogue

// Results to memory.  A lane holds row l % 16, columns 4 (l / 16) + 0..3 of
// each fragment; through LDS (each wave in its own region, RC rows at a time)
// it gets 8 consecutive columns of one row instead, so that bias, residual and
// results are read and written in 16-byte pieces of whole lines.  Everything is
// fp32 up to the one rounding to the output.
//   out: the tile's first row; left: rows there; e: expert of the bias;
//   c0: first result column of the tile
template <typename TILE, bool GATED, bool EPILOGUE>
__device__ __forceinline__ void linear_store(char *lds, const LinearArgs &a, float4v (&acc)[TILE::FP][TILE::FQ], int e,
                                             int64_t row0, int left, int c0, int n, uint16_t *out, int64_t so)
{
    constexpr int FP = TILE::FP, FQ = TILE::FQ, RC = TILE::RC, WJ = TILE::WJ;
    constexpr int OJ = GATED ? WJ / 2 : WJ;          // result columns of a wave
    constexpr int LPR = OJ / 8, RPP = 64 / LPR, PASSES = RC / RPP;
    const int wave = uniform(threadIdx.x >> 6), wp = wave / TILE::WN, wq = wave % TILE::WN;
    const int lane = threadIdx.x & 63, fr = lane & 15, fk = lane >> 4, pr = lane / LPR, pc = lane % LPR;
    const int c = c0 + wq * OJ + pc * 8;
    // columns in LDS of this lane's (gate's) eight, in fragments of 16
    const int lc = GATED ? (pc >> 1) * 32 + (pc & 1) * 8 : pc * 8;
    float *wide = reinterpret_cast<float *>(lds) + wave * RC * WJ;
    auto wswap = [](int r) { return WJ == 64 ? r & 15 : (r >> 1) & 7; };
    float bias[2][8];
    if constexpr (EPILOGUE) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool there = a.bias && c + k < n;
            bias[0][k] = there ? bias_at(a.bias, a.bias_f32, e * a.sb + c + k) : 0.0f;
            if (GATED)
                bias[1][k] = there ? bias_at(a.bias, a.bias_f32, e * a.sb + n + c + k) : 0.0f;
        }
    }
    wait_stage<0>();  // every wave is done with the stages
#pragma unroll
    for (int ic = 0; ic < FP * 16; ic += RC) {
#pragma unroll
        for (int i = 0; i < RC / 16; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j)
                *reinterpret_cast<float4v *>(wide + (i * 16 + fr) * WJ + ((4 * j + fk) ^ wswap(i * 16 + fr)) * 4) =
                    acc[ic / 16 + i][j];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + pr, i = wp * FP * 16 + ic + r;
            if (i >= left || c >= n)
                continue;
            auto read = [&](int col, float (&v)[8]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4v x = *reinterpret_cast<const float4v *>(wide + r * WJ + ((col / 4 + h) ^ wswap(r)) * 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[4 * h + k] = x[k];
                }
            };
            float v[8];
            read(lc, v);
            if constexpr (EPILOGUE) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] += bias[0][k];
                if (a.pre)
                    store8(a.pre + (row0 + i) * a.spre, c, n, v);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = act_value(a.act, v[k]);
                if constexpr (GATED) {
                    float g[8];
                    read(lc + 16, g);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[k] += bias[1][k];
                    if (a.pre)
                        store8(a.pre + (row0 + i) * a.spre + n, c, n, g);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] *= g[k];
                }
                if (a.resid) {
                    const Piece<uint16_t> x = load8(a.resid + (row0 + i) * a.sr, c, n);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] += x.get(k);
                }
            }
            store8(out + (row0 + i) * so, c, n, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// zeros for the rows of no group
template <int TM, int TN, int THREADS>
__device__ __forceinline__ void clear_tile(uint16_t *out, int64_t so, int64_t row0, int left, int c0, int n)
{
    constexpr int PPR = TN / 8;
    const float zero[8] = {};
    for (int at = threadIdx.x; at < TM * PPR; at += THREADS) {
        const int r = at / PPR, c = c0 + (at % PPR) * 8;
        if (r < left && c < n)
            store8(out + (row0 + r) * so, c, n, zero);
    }
}

// ---------------------------------------------------------------- kernels

// One tile per workgroup.
template <int MODE, typename TILE, bool GATED, bool MX>
__global__ __launch_bounds__(TILE::THREADS, 2) void linear_kernel(LinearArgs a)
{
    constexpr bool PT = MODE == kGradW, QT = MODE != kForward;
    typedef LinearStages<TILE, PT, QT, MX> S;
    __shared__ __attribute__((aligned(16))) char lds[TILE::NST * S::BYTES];
    constexpr int TM = TILE::TM, TN = TILE::TN, TJ = GATED ? TN / 2 : TN;
    const int tn = (a.n + TJ - 1) / TJ;
    int e, i0, c0, left, k;
    int64_t row0;
    if constexpr (MODE == kGradW) {
        // every expert's (wide, width) result; the sum runs over the group's rows
        const int tm = (a.wide + TM - 1) / TM, total = a.experts * tm * tn, t = spread(blockIdx.x, total);
        if (t >= total)
            return;
        e = t / (tm * tn);
        int bi, bj, start;
        band_tile(t % (tm * tn), tm, tn, bi, bj);
        group_rows(a.offs, a.experts, a.rows, e, start, k);
        row0 = uniform(start);
        k = uniform(k);
        i0 = bi * TM;
        c0 = bj * TN;
        left = a.wide - i0;
    } else {
        const int tm = count_row_tiles<TM>(a), total = tm * tn, t = spread(blockIdx.x, total);
        if (t >= total)
            return;
        int bi, bj, r0;
        band_tile(t, tm, tn, bi, bj);
        find_row_tile<TM>(a, bi, e, r0, left);
        row0 = r0;
        i0 = 0;
        c0 = bj * TJ;
        if (e >= a.experts) {
            clear_tile<TM, TJ, TILE::THREADS>(a.out, a.so, row0, left, c0, a.n);
            if (MODE == kForward && a.pre) {
                clear_tile<TM, TJ, TILE::THREADS>(a.pre, a.spre, row0, left, c0, a.n);
                if (GATED)
                    clear_tile<TM, TJ, TILE::THREADS>(a.pre + a.n, a.spre, row0, left, c0, a.n);
            }
            return;
        }
        k = MODE == kForward ? a.width : a.wide;
    }

    S st;
    st.lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    // bytes of k of one row, in whole chunks: rows whose length is not are padded
    const int kb = MX ? k : 2 * ((k + 7) & ~7);
    st.stages = MODE == kGradW ? (k + 63) / 64 : (kb + kRowBytes - 1) / kRowBytes;
    st.live = MODE == kGradW ? 8 : ((kb - 1) % kRowBytes + 16) / 16;
    if constexpr (MODE == kGradW) {
        st.p.set_turned(a.p + row0 * a.ldp + (int64_t)i0 * 2, a.ldp, (uint32_t)(((a.wide + 7) & ~7) - i0) * 2, k);
        st.q.set_turned(a.q + row0 * a.ldq + (int64_t)c0 * 2, a.ldq, (uint32_t)(((a.n + 7) & ~7) - c0) * 2, k);
    } else {
        const int rows = min(left, TM);
        st.p.set_rows(a.p + row0 * a.ldp, a.ldp, (uint32_t)((rows - 1) * a.ldp) + kb, [&](int r) { return r < rows ? r : -1; });
        const char *q = a.q + e * a.qe;
        if constexpr (QT) {
            st.q.set_turned(q + (int64_t)c0 * 2, a.ldq, (uint32_t)(((a.n + 7) & ~7) - c0) * 2, a.wide);
        } else {
            // tile row r: gated, fragments of 16 rows of the gate and of the
            // value in turn
            const int n = a.n - c0;
            auto row = [&](int r) {
                const int at = GATED ? (r >> 5) * 16 + (r & 15) : r;
                return at >= n ? -1 : GATED && (r & 16) ? at + a.n : at;
            };
            const int last = GATED ? a.wide - 1 - c0 : min(n, TN) - 1;
            st.q.set_rows(q + c0 * a.ldq, a.ldq, (uint32_t)(last * a.ldq) + kb, row);
            if constexpr (MX) {
                const int t = threadIdx.x, r = row(min(max(t - TM, 0), TN - 1));
                st.scales = t < TM ? a.sp + (row0 + min(t, rows - 1)) * a.ldsp
                                   : a.sq + e * a.sqe + (int64_t)(c0 + max(r, 0)) * a.ldsq;
            }
        }
    }
    float4v acc[TILE::FP][TILE::FQ];
#pragma unroll
    for (int i = 0; i < TILE::FP; ++i)
#pragma unroll
        for (int j = 0; j < TILE::FQ; ++j)
            acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    const int wave = uniform(threadIdx.x >> 6), r0 = wave / TILE::WN * TILE::FP * 16, q0 = wave % TILE::WN * TILE::FQ * 16;
    if (st.stages > 0)
        linear_pipeline<TILE, PT, QT, MX>(st, r0, q0, acc);
    uint16_t *out = MODE == kGradW ? a.out + e * a.oe : a.out;
    linear_store<TILE, GATED, MODE == kForward>(lds, a, acc, e, MODE == kGradW ? i0 : row0, left, c0, a.n, out, a.so);
}

// ---------------------------------------------------------------- around them

// (count, rows, cols) elements of bf16 in rows padded with zeros to `padded`
// elements (a multiple of 8), for operands whose rows do not start on 16 bytes
// or whose length is no multiple of 8.
__global__ __launch_bounds__(256) void linear_pack_kernel(const uint16_t *__restrict__ in, int64_t se, int64_t sr,
                                                          int rows, int cols, uint16_t *__restrict__ out, int padded)
{
    const int pieces = padded / 8;
    const uint16_t *src = in + blockIdx.y * se;
    uint16_t *dst = out + (int64_t)blockIdx.y * rows * padded;
    const int64_t all = (int64_t)rows * pieces;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (int64_t)gridDim.x * 256) {
        const int64_t r = at / pieces;
        const int c = (int)(at % pieces) * 8;
        st_piece<uint16_t>(dst + r * padded + c, load8(src + r * sr, c, cols));
    }
}

// rows of scales in whole words
__global__ __launch_bounds__(256) void linear_pack_scales_kernel(const uint8_t *__restrict__ in, int64_t se,
                                                                 int64_t sr, int64_t sb, int rows, int blocks,
                                                                 uint8_t *__restrict__ out, int padded)
{
    const int words = padded / 4;
    const uint8_t *src = in + blockIdx.y * se;
    uint8_t *dst = out + (int64_t)blockIdx.y * rows * padded;
    const int64_t all = (int64_t)rows * words;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (int64_t)gridDim.x * 256) {
        const int64_t r = at / words;
        const int c = (int)(at % words) * 4;
        uint32_t v = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v |= (c + k < blocks ? (uint32_t)src[r * sr + (c + k) * sb] : 0u) << (8 * k);
        *reinterpret_cast<uint32_t *>(dst + r * padded + c) = v;
    }
}

// dz from dy and the saved z (PRE), and the columns' sums over each group in
// parts of kSliceRows rows.
//   plain  dz = dy act'(z)        gated  dz = [dy value act'(gate), dy act(gate)]
// dz is rounded to bf16, the type that the two products take; the sums are of
// the values before that rounding.  A wave has every fourth row of a slice and
// 512 columns.
constexpr int kSliceRows = 64;

template <bool GATED, bool PRE>
__global__ __launch_bounds__(256) void linear_dact_kernel(LinearArgs a, const uint16_t *__restrict__ dy, int64_t sy,
                                                          const uint16_t *__restrict__ pre, int64_t spre,
                                                          uint16_t *dz, int64_t sdz, float *parts)
{
    __shared__ float sums[4][GATED ? 2 : 1][512];
    const int slices = count_row_tiles<kSliceRows>(a);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = GATED ? a.wide / 2 : a.wide;
    const int c = blockIdx.y * 512 + lane * 8;
    for (int s = blockIdx.x; s < slices; s += gridDim.x) {
        int e, row0, left;
        find_row_tile<kSliceRows>(a, s, e, row0, left);
        if (e >= a.experts)
            return;  // and so are all slices after it
        const int end = min(left, kSliceRows);
        float total[GATED ? 2 : 1][8] = {};
        for (int r = wave; r < end && c < n; r += 4) {
            const int64_t row = (int64_t)row0 + r;
            const Piece<uint16_t> d = load8(dy + row * sy, c, n);
            float g[8], v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                g[k] = d.get(k);
            if constexpr (PRE) {
                const Piece<uint16_t> z = load8(pre + row * spre, c, n);
                uint16_t *to = dz + row * sdz;
                if constexpr (GATED) {
                    const Piece<uint16_t> w = load8(pre + row * spre + n, c, n);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        v[k] = g[k] * act_value(a.act, z.get(k));
                        g[k] = g[k] * w.get(k) * act_slope(a.act, z.get(k));
                    }
                    store8(to, c, n, g);
                    store8(to + n, c, n, v);
                    if (c + 8 >= n)
                        for (int k = 2 * n; k < sdz; ++k)  // the padding
                            to[k] = 0;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[k] *= act_slope(a.act, z.get(k));
                    if (c + 8 > n)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            g[k] = c + k < n ? g[k] : 0.0f;
                    store8(to, c, (int)sdz, g);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                total[0][k] += g[k];
                if constexpr (GATED)
                    total[1][k] += v[k];
            }
        }
        if (!parts)
            continue;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sums[wave][h][lane * 8 + k] = total[h][k];
        __syncthreads();
        for (int at = threadIdx.x; at < (GATED ? 1024 : 512); at += 256) {
            const int h = at >> 9, col = at & 511, to = blockIdx.y * 512 + col;
            if (to < n)
                parts[(int64_t)s * a.wide + h * n + to] =
                    (sums[0][h][col] + sums[1][h][col]) + (sums[2][h][col] + sums[3][h][col]);
        }
    }
}

// The slices' sums of each group, in order, in fp64.
__global__ __launch_bounds__(256) void linear_bias_kernel(LinearArgs a, const float *__restrict__ parts,
                                                          float *__restrict__ out)
{
    const int e = blockIdx.y;
    int before = 0, own = 0, start, len;
    for (int g = threadIdx.x & 63; g <= e; g += 64) {
        group_rows(a.offs, a.experts, a.rows, g, start, len);
        const int n = (len + kSliceRows - 1) / kSliceRows;
        (g < e ? before : own) += n;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        before += __shfl_xor(before, m, 64);
        own += __shfl_xor(own, m, 64);
    }
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.wide)
        return;
    double s = 0.0;
    for (int i = 0; i < own; ++i)
        s += parts[(int64_t)(before + i) * a.wide + c];
    out[(int64_t)e * a.wide + c] = (float)s;
}

}  // namespace mxq
