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

#include <type_traits>

#include "linear_ops.hpp"
#include "moe_rows_kernels.hpp"
#include "mxq_device.hpp"
#include "stream_ops.hpp"
#include "tile_ops.hpp"
#include "wave_ops.hpp"

namespace mxq {

enum LinearMode { kForward, kGradX, kGradW };
// Operands: bf16, or MXFP8 with the scales of a row in whole words, or of any
// strides.
enum LinearFormat { kBf16, kMxWords, kMxBytes };
// Operands and results of a call; leading strides in bytes for what is read
// into LDS, else in elements.
struct LinearArgs {
    const char *p, *q;            // see the modes
    int64_t ldp, ldq, qe;         // qe: from expert to expert
    const uint8_t *sp, *sq;       // e8m0 scales (MXFP8)
    int64_t ldsp, ldsq, sqe;
    int64_t sbp, sbq;             // from block to block (kMxWords: 1)
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
    float *parts;                 // sums in parts: (splits, result rows, ldparts), rows of whole 8
    int64_t ldparts, part_size;   // part_size: from part to part
    int splits;
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
    return uniform(((s / run) * 8 + (block & 7)) * run + s % run);
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
};

// one workgroup of eight alternating waves per CU, 128 KB of LDS
using LinearLarge = LinearTile<256, 256, 2, 4, 2>;
using LinearHalf = LinearTile<256, 128, 2, 4, 2>;

// k of a stage
constexpr int kRowBytes = 128;

// One operand of a tile: EXT rows of 128 bytes of k; or turned, EXT / 64 blocks
// of 64 rows of k, 64 elements (128 bytes) of bf16 each.  THREADS threads.
//
// Loads into LDS are linear, so a load is whole rows or a whole block's; to
// spread the lanes of one LDS read over the banks, the order of the chunks of a
// row is exchanged in the addresses that are loaded: 16-byte chunk c of row r is
// at c ^ rswap(r), 32-byte chunk c of a turned row k at c ^ tswap(k).
template <int EXT, int THREADS, bool TURNED>
struct Panel {
    static constexpr int RPL = THREADS / 8;               // rows per load
    static constexpr int LOADS = EXT / RPL;
    static_assert(RPL % 16 == 0 && 64 % RPL == 0, "the chunk orders repeat with each load");
    const char *base;
    int64_t step;                 // bytes from stage to stage
    int64_t ld;
    uint32_t off[LOADS];          // of this thread's chunks
    uint32_t range;               // bytes from base on (rows), of a row (turned)
    int rows;                     // turned: rows from base on
    int chunk;                    // this thread's chunk of k

    static __device__ __forceinline__ int rswap(int r) { return (r >> 1) & 7; }
    static __device__ __forceinline__ int tswap(int k) { return ((k >> 1) & 1) | ((k >> 3) & 1) << 1; }

    // row(r): the operand's row that tile row r holds, relative to base, or -1
    template <typename Row>
    __device__ __forceinline__ void set_rows(const char *b, int64_t stride, uint32_t bytes, Row &&row)
    {
        base = b;
        ld = stride;
        step = kRowBytes;
        range = bytes;
        rows = 0;
        const int r = threadIdx.x / 8;
        chunk = (threadIdx.x % 8) ^ rswap(r);
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
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int r = threadIdx.x / 8 + u * RPL, k = r % 64;
            const uint32_t c = (r / 64) * 128 + ((threadIdx.x % 8) ^ (tswap(k) << 1)) * 16;
            // a row shorter than the tile: not the next row's start, where
            // that may be past the last row
            off[u] = c < bytes ? (uint32_t)(k * (uint32_t)stride + c) : 0x80000000u;
        }
    }

    __device__ __forceinline__ void skip(int stages)
    {
        base += stages * step;
        if (TURNED)
            rows -= stages * 64;
        else
            range -= (uint32_t)(stages * kRowBytes);
    }

    // load u of stage kt to lds + 16 * thread; `live`: chunks of k of the stage
    __device__ __forceinline__ void load(int u, int kt, int live, uint32_t lds) const
    {
        const uint32_t bytes = TURNED ? (uint32_t)((min(rows - kt * 64, 64) - 1) * ld) + range
                                      : range - (uint32_t)(kt * kRowBytes);
        // uniform all of it, but not provably so: without this the load becomes
        // a loop over the lanes' descriptors
        const uint64_t at = (uint64_t)(uintptr_t)base + (uint64_t)(kt * step);
        const uint64_t from = (uint32_t)uniform((int)at) | (uint64_t)(uint32_t)uniform((int)(at >> 32)) << 32;
        __amdgpu_buffer_rsrc_t rs = buffer_rsrc(reinterpret_cast<const void *>(from), (uint32_t)uniform((int)bytes));
        uint32_t o = off[u];
        if (!TURNED && live < 8)
            o = chunk < live ? o : 0x80000000u;
        const uint32_t dst = lds + (uint32_t)(u * THREADS + (threadIdx.x & ~63)) * 16;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void *)(uintptr_t)uniform((int)dst), 16, (int)o, 0, 0, 0);
    }

    // LDS addresses of this lane's fragment reads, from tile row (or column)
    // `first`, a multiple of 16 N, on; the rest of an address is a constant of
    // the instruction
    template <int N>
    struct Reads {
        static constexpr int A = TURNED ? (N < 4 ? N : 4) : 2;
        uint32_t a[A];
        __device__ __forceinline__ Reads(uint32_t lds, int first)
        {
            const int fr = threadIdx.x & 15, fk = (threadIdx.x & 63) >> 4;
            if constexpr (TURNED) {
                const int kr = 8 * fk + (fr >> 2);  // and the four rows after
#pragma unroll
                for (int i = 0; i < A; ++i)
                    a[i] = lds + (uint32_t)((first / 64) * 8192 + kr * 128 + ((first / 16 + i) % 4 ^ tswap(kr)) * 32 + (fr & 3) * 8);
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
                    const uint32_t b = a[(I0 + i) % A] + at + (I0 + i) / 4 * 8192 + h * 4096;
                    const half4 x = read_transposed(b), y = read_transposed(b + 512);
                    f[i] = half8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                } else {
                    f[i] = read_lds(a[h] + at + (I0 + i) * 16 * 128);
                }
            }
        }
    };
};

// acc += P Q over a stage, fragments I0.. of P.  Q is the first operand: a
// lane's four results lie along j.  The scaled product takes both halves of a
// stage at once (128 values of k): lane 16 b + i holds bytes 16 b and 64 + 16 b
// of row i and supplies the scale of its 32-value block b.
template <int F, int I0, int N, int FP, int FQ>
__device__ __forceinline__ void multiply_stage(const half8 (&p0)[N], const half8 (&p1)[N], const half8 (&q0)[FQ],
                                               const half8 (&q1)[FQ], const int (&sp)[FP], const int (&sq)[FQ],
                                               float4v (&acc)[FP][FQ])
{
    if constexpr (F != kBf16) {
        // both halves of a fragment
        auto whole = [](const half8 &x, const half8 &y) {
            typedef int int4v __attribute__((ext_vector_type(4)));
            const int4v u = __builtin_bit_cast(int4v, x), v = __builtin_bit_cast(int4v, y);
            return int8v{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
        };
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j)
                acc[I0 + i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    whole(q0[j], q1[j]), whole(p0[i], p1[i]), acc[I0 + i][j], 0, 0, 0, sq[j], 0, sp[I0 + i]);
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
// four blocks per row and stage in LDS, or a byte per lane and fragment straight
// into registers.  Bytes spare the small tiles a pass that lays the scales out in
// words: 27 rows over 23 experts of 72 x 96 12.8 us a call (23.7 with it), sums over
// 2080 as long as with it.
template <typename TILE, bool PT, bool QT, int F>
struct LinearStages {
    typedef Panel<TILE::TM, TILE::THREADS, PT> PanelP;
    typedef Panel<TILE::TN, TILE::THREADS, QT> PanelQ;
    static constexpr int LP = PanelP::LOADS, LQ = PanelQ::LOADS, LS = F == kMxWords ? (TILE::TM + TILE::TN + TILE::THREADS - 1) / TILE::THREADS : 0;
    static constexpr int LOADS = LP + LQ + LS;
    static constexpr int BYTES = TILE::STAGE + LS * TILE::THREADS * 4;
    PanelP p;
    PanelQ q;
    const uint8_t *scales[LS > 0 ? LS : 1];  // words: this thread's rows
    // bytes: the rows of this lane in each fragment, the stride from block to
    // block, and how many blocks there are
    const uint8_t *byte_p[F == kMxBytes ? TILE::FP : 1], *byte_q[F == kMxBytes ? TILE::FQ : 1];
    int64_t stride_p, stride_q;
    int blocks;
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
            const int l = u - LP - LQ;
            const uint32_t dst = at + TILE::STAGE + (l * TILE::THREADS + (threadIdx.x & ~63)) * 4;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(scales[l] + kt * 4),
                                             (__attribute__((address_space(3))) void *)(uintptr_t)uniform((int)dst), 4, 0, 0);
        }
    }
    __device__ __forceinline__ void load(int s, int kt) const
    {
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
            load_one(s, u, kt);
    }

    // stages [first, last) alone
    __device__ __forceinline__ void part(int first, int last)
    {
        p.skip(first);
        q.skip(first);
        if constexpr (F == kMxWords)
#pragma unroll
            for (int l = 0; l < LS; ++l)
                scales[l] += first * 4;
        if constexpr (F == kMxBytes) {
#pragma unroll
            for (int i = 0; i < TILE::FP; ++i)
                byte_p[i] += first * 4 * stride_p;
#pragma unroll
            for (int i = 0; i < TILE::FQ; ++i)
                byte_q[i] += first * 4 * stride_q;
            blocks -= first * 4;
        }
        live = last < stages ? 8 : live;
        stages = last - first;
    }

    // scales of N fragments from tile row `first` on (of Q: TM further), each
    // lane its block's in the lowest byte; blocks past k are zeros in memory
    template <int N>
    __device__ __forceinline__ void read_scales(int s, int first, int (&v)[N]) const
    {
        if constexpr (F == kMxWords) {
            const int fr = threadIdx.x & 15, fk = (threadIdx.x & 63) >> 4;
            const uint32_t a = lds0 + s * BYTES + TILE::STAGE + (uint32_t)(first + fr) * 4;
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = *(__attribute__((address_space(3))) const int *)(uintptr_t)(a + i * 64) >> (8 * fk);
        }
    }

    // bytes: those of stage kt; a block past the last one counts as zero (its
    // values are, and a scale that is none must not make them NaN)
    __device__ __forceinline__ void load_scales(int kt, int (&sp)[TILE::FP], int (&sq)[TILE::FQ]) const
    {
        if constexpr (F == kMxBytes) {
            const int own = kt * 4 + ((threadIdx.x & 63) >> 4), b = min(own, blocks - 1);
#pragma unroll
            for (int i = 0; i < TILE::FP; ++i)
                sp[i] = byte_p[i][b * stride_p];
#pragma unroll
            for (int i = 0; i < TILE::FQ; ++i)
                sq[i] = byte_q[i][b * stride_q];
            if (own >= blocks) {
#pragma unroll
                for (int i = 0; i < TILE::FP; ++i)
                    sp[i] = 0;
#pragma unroll
                for (int i = 0; i < TILE::FQ; ++i)
                    sq[i] = 0;
            }
        }
    }
};

// Fragments are read one stage ahead of their MFMAs.  At a stage's one barrier
// every wave has read stage kt and has stage kt + 1; the load of stage kt + NST
// overwrites stage kt.
template <typename TILE, bool PT, bool QT, int F>
__device__ __forceinline__ void linear_pipeline(const LinearStages<TILE, PT, QT, F> &st, int row0, int col0,
                                                float4v (&acc)[TILE::FP][TILE::FQ])
{
    typedef LinearStages<TILE, PT, QT, F> S;
    constexpr int NST = TILE::NST, FP = TILE::FP, FQ = TILE::FQ;
    const typename S::PanelP::template Reads<FP> rp(st.lds0, row0);
    const typename S::PanelQ::template Reads<FQ> rq(st.lds0 + TILE::TM * 128, col0);
    struct Frags {
        half8 p0[FP], p1[FP], q0[FQ], q1[FQ];
        int sp[FP], sq[FQ];
    } f[2];
    auto read = [&](int s, Frags &x) {
        const uint32_t at = s * S::BYTES;
        rq.template read<0>(at, 0, x.q0);
        rp.template read<0>(at, 0, x.p0);
        rq.template read<0>(at, 1, x.q1);
        rp.template read<0>(at, 1, x.p1);
        st.read_scales(s, row0, x.sp);
        st.read_scales(s, TILE::TM + col0, x.sq);
    };
    const int end = st.stages;
    st.load_scales(0, f[0].sp, f[0].sq);
    for (int s = 0; s < NST; ++s)
        if (s < end)
            st.load(s, s);
    if (end >= NST)
        wait_stage<(NST - 1) * S::LOADS>();
    else
        wait_stage<0>();
    read(0, f[0]);
    int now = 0, kt = 0;
    auto step = [&](Frags &x, Frags &y) {
        const int next = now + 1 == NST ? 0 : now + 1;
        if (kt + 1 < end) {
            if (kt + NST <= end)
                wait_stage<(NST - 2) * S::LOADS>();
            else
                wait_stage<0>();
            // loads return in order: before those of a later stage
            st.load_scales(kt + 1, y.sp, y.sq);
            if (kt + NST < end)
                st.load(now, kt + NST);
            read(next, y);
        }
        multiply_stage<F, 0>(x.p0, x.p1, x.q0, x.q1, x.sp, x.sq, acc);
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

// Two groups of four waves, one wave of each on every SIMD, one phase apart:
// while one group's MFMAs run the other reads its fragments.  Group 0 has the
// upper half of the tile's rows, group 1 the lower; each half's rows are taken
// in two quarters.  A stage takes four phases with a barrier after each:
//   ra  read Q, all scales and the first quarter     ma  multiply
//   rb  read the second quarter                      mb  multiply
// and group 1 is in the phase before group 0's.
//
// Two stages in LDS, but a stage's parts are loaded as soon as the part that
// they overwrite has been read by both groups (a read phase ends with its
// reads returned), so every part has five phases to arrive.  In either group's
// phases of stage t:
//   ra(t)  quarters 1 and 3 of t + 1             (first read in rb(t + 1))
//   rb(t)  Q, scales, quarters 0 and 2 of t + 2  (first read in ra(t + 2))
// The loads of a wave return in order: at the end of group 0's mb(t) the parts
// for ra(t + 1) have landed when only those issued since are pending, 2 of t + 1
// and the FIRST of t + 2, at the end of its ma(t) those for rb(t) when again as
// many are.
template <typename TILE, bool PT, bool QT, int F>
struct LinearAlternating {
    typedef LinearStages<TILE, PT, QT, F> S;
    static_assert(TILE::NST == 2 && TILE::WM == 2 && TILE::WN == 4 && TILE::TM == 256 && S::LP == 4,
                  "loads 0-3 are the quarters, the rest Q and the scales");
    static constexpr int FP = TILE::FP, FQ = TILE::FQ, H = FP / 2;
    static constexpr int FIRST = S::LOADS - 2;
    const S &st;
    const typename S::PanelP::template Reads<FP> rp;
    const typename S::PanelQ::template Reads<FQ> rq;
    int row0, col0;
    half8 p0[H], p1[H], q0[FQ], q1[FQ];
    int sp[FP], sq[FQ];

    __device__ __forceinline__ LinearAlternating(const S &s, int r, int c)
        : st(s), rp(s.lds0, r), rq(s.lds0 + TILE::TM * 128, c), row0(r), col0(c)
    {
    }

    static __device__ __forceinline__ void load_a(const S &st, int kt)
    {
#pragma unroll
        for (int u = 4; u < S::LOADS; ++u)
            st.load_one(kt & 1, u, kt);
        st.load_one(kt & 1, 0, kt);
        st.load_one(kt & 1, 2, kt);
    }
    __device__ __forceinline__ void load_b(int kt) const
    {
        st.load_one(kt & 1, 1, kt);
        st.load_one(kt & 1, 3, kt);
    }
    __device__ __forceinline__ void read_a(int kt)
    {
        const uint32_t at = (kt & 1) * S::BYTES;
        rq.template read<0>(at, 0, q0);
        rp.template read<0>(at, 0, p0);
        rq.template read<0>(at, 1, q1);
        rp.template read<0>(at, 1, p1);
        st.read_scales(kt & 1, row0, sp);
        st.read_scales(kt & 1, TILE::TM + col0, sq);
    }
    __device__ __forceinline__ void read_b(int kt)
    {
        const uint32_t at = (kt & 1) * S::BYTES;
        rp.template read<H>(at, 0, p0);
        rp.template read<H>(at, 1, p1);
    }
    template <int I0>
    __device__ __forceinline__ void products(float4v (&acc)[FP][FQ])
    {
        __builtin_amdgcn_s_setprio(1);
        multiply_stage<F, I0>(p0, p1, q0, q1, sp, sq, acc);
        __builtin_amdgcn_s_setprio(0);
    }

    // one stage; MORE: how many stages follow (0, 1, or 2 for two and more)
    template <bool LATER, int MORE>
    __device__ __forceinline__ void stage(int kt, float4v (&acc)[FP][FQ])
    {
        constexpr int kB = MORE >= 1 ? 2 + FIRST : 0;                         // pending when rb may begin
        constexpr int kNext = MORE >= 2 ? 2 + FIRST : MORE == 1 ? 2 : -1;     // when the next ra may
        read_a(kt);
        if (MORE >= 1)
            load_b(kt + 1);
        phase_end<LATER ? kB : -1>();
        products<0>(acc);
        phase_end<LATER ? -1 : kB>();
        read_b(kt);
        if (MORE >= 2)
            load_a(st, kt + 2);
        phase_end<LATER ? kNext : -1>();
        products<H>(acc);
        phase_end<LATER ? -1 : kNext>();
    }

    template <bool LATER>
    __device__ __forceinline__ void run_group(float4v (&acc)[FP][FQ])
    {
        if (LATER)
            phase_end<-1>();
        const int end = st.stages;
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

    // what is on its way before run(); the stages are free
    static __device__ __forceinline__ void first_loads(const S &st)
    {
        st.load(0, 0);
        if (st.stages > 1)
            load_a(st, 1);
    }

    // Waits for whatever was issued after first_loads, too.  At the end every
    // wave has read every stage: the last read phase of either group is before
    // the last barrier.
    __device__ __forceinline__ void run(float4v (&acc)[FP][FQ])
    {
        phase_end<0>();
        if (row0 != 0)
            run_group<true>(acc);
        else
            run_group<false>(acc);
    }
};

// Rows of 16 lanes: a's second and fourth change places with b's first and
// third.
__device__ __forceinline__ void swap_rows(float &a, float &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}

// Results to memory.  A lane holds row l % 16, columns 4 (l / 16) + 0..3 of each
// fragment.  Two fragments change lane rows, and each lane has 8 consecutive
// columns of one of them: bias, residual and results are read and written in
// 16-byte pieces, 64 bytes of a row at a time, without LDS and without meeting
// the other waves.  Everything is fp32 up to the one rounding to the output.
//   row0: first row of the tile in the results; left: rows there; e: expert of
//   the bias; c0: first result column of the tile
template <typename TILE, bool GATED, bool EPILOGUE>
__device__ __forceinline__ void linear_store(const LinearArgs &a, float4v (&acc)[TILE::FP][TILE::FQ], int e,
                                             int64_t row0, int left, int c0, int n, uint16_t *out, int64_t so)
{
    constexpr int FP = TILE::FP, FQ = TILE::FQ;
    // the pairs of fragments: next to one another along j, of a gate two
    // further (the value between); with one gate fragment along i
    constexpr bool ALONG_I = GATED && FQ == 2;
    constexpr int PAIRS = ALONG_I ? 1 : GATED ? FQ / 4 : FQ / 2;
    const int wave = uniform(threadIdx.x >> 6), wp = wave / TILE::WN, wq = wave % TILE::WN;
    const int lane = threadIdx.x & 63, fr = lane & 15, fk = lane >> 4;
    const int r0 = wp * FP * 16 + fr + (ALONG_I ? (fk & 1) * 16 : 0);
    const int w0 = c0 + wq * (GATED ? FQ * 8 : FQ * 16) + (fk >> 1) * 8 + (ALONG_I ? 0 : (fk & 1) * 16);
    float bias[PAIRS][GATED ? 2 : 1][8];
    if constexpr (EPILOGUE) {
#pragma unroll
        for (int p = 0; p < PAIRS; ++p)
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int c = w0 + p * 32 + k;
                    bias[p][h][k] = a.bias && c < n ? bias_at(a.bias, a.bias_f32, e * a.sb + h * n + c) : 0.0f;
                }
    }
    // eight values of one fragment from its pair
    auto join = [](float4v x, float4v y, float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo = x[k], hi = y[k];
            swap_rows(lo, hi);
            v[k] = lo;
            v[4 + k] = hi;
        }
    };
    Piece<uint16_t> resid[2][PAIRS];
    auto load_resid = [&](int i, int set) {
        if constexpr (EPILOGUE) {
            if (a.resid) {
                const int r = r0 + i * 16;
#pragma unroll
                for (int p = 0; p < PAIRS; ++p)
                    if (r < left && w0 + p * 32 < n)
                        resid[set][p] = load8(a.resid + (row0 + r) * a.sr, w0 + p * 32, n);
            }
        }
    };
    constexpr int STEP = ALONG_I ? 2 : 1;
    load_resid(0, 0);
#pragma unroll
    for (int i = 0; i < FP; i += STEP) {
        if (i + STEP < FP)
            load_resid(i + STEP, (i / STEP + 1) & 1);
        const int r = r0 + i * 16;
        const int64_t row = row0 + r;
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            const int c = w0 + p * 32;
            float v[8], g[8];
            if constexpr (ALONG_I) {
                join(acc[i][0], acc[i + 1][0], v);
                join(acc[i][1], acc[i + 1][1], g);
            } else if constexpr (GATED) {
                join(acc[i][4 * p], acc[i][4 * p + 2], v);
                join(acc[i][4 * p + 1], acc[i][4 * p + 3], g);
            } else {
                join(acc[i][2 * p], acc[i][2 * p + 1], v);
            }
            if (r >= left || c >= n)
                continue;
            if constexpr (EPILOGUE) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] += bias[p][0][k];
                if (a.pre)
                    store8(a.pre + row * a.spre, c, n, v);
                act_values(a.act, v);
                if constexpr (GATED) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[k] += bias[p][1][k];
                    if (a.pre)
                        store8(a.pre + row * a.spre + n, c, n, g);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] *= g[k];
                }
                if (a.resid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] += resid[(i / STEP) & 1][p].get(k);
                }
            }
            store8(out + row * so, c, n, v);
        }
    }
}

// The sums of a part as they are, for linear_join_kernel: whole pieces of four
// columns, a gate's value half a row further.
template <typename TILE, bool GATED>
__device__ __forceinline__ void store_part(const LinearArgs &a, float4v (&acc)[TILE::FP][TILE::FQ], int64_t row0, int left,
                                           int c0, int n, float *out)
{
    constexpr int FP = TILE::FP, FQ = TILE::FQ;
    const int wave = uniform(threadIdx.x >> 6), wp = wave / TILE::WN, wq = wave % TILE::WN;
    const int lane = threadIdx.x & 63, fr = lane & 15, fk = lane >> 4;
#pragma unroll
    for (int i = 0; i < FP; ++i) {
        const int r = wp * FP * 16 + i * 16 + fr;
        float *row = out + (row0 + r) * a.ldparts;
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const int f = wq * FQ + j, c = c0 + (GATED ? f / 2 : f) * 16 + 4 * fk;
            if (r >= left || c >= n)
                continue;
            *reinterpret_cast<float4v *>(row + (GATED && (f & 1) ? a.ldparts / 2 : 0) + c) = acc[i][j];
        }
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

// A tile of the results.
struct TileAt {
    int e;                // its expert; `experts`: rows of no group, to clear
    int i0, c0;           // grad W: first row of dW; first result column
    int left;             // result rows from the tile's first on
    int k;                // length of the sum
    int64_t row0;         // first row among the tokens
};

template <int MODE, typename TILE, bool GATED>
struct LinearGrid {
    static constexpr int TM = TILE::TM, TJ = GATED ? TILE::TN / 2 : TILE::TN;
    int tm, tn, total;
    __device__ __forceinline__ LinearGrid(const LinearArgs &a)
    {
        tn = (a.n + TJ - 1) / TJ;
        tm = MODE == kGradW ? (a.wide + TM - 1) / TM : count_row_tiles<TM>(a);
        total = MODE == kGradW ? a.experts * tm * tn : tm * tn;
    }
    __device__ __forceinline__ TileAt at(const LinearArgs &a, int t) const
    {
        // uniform(): divisions come out of vector registers, and from there a
        // descriptor would be made for each lane
        TileAt x;
        int bi, bj, e, row0, left;
        if constexpr (MODE == kGradW) {
            // every expert's (wide, width) result; the sum runs over the group's rows
            e = uniform(t / (tm * tn));
            band_tile(uniform(t - e * tm * tn), tm, tn, bi, bj);
            bi = uniform(bi);
            int len;
            group_rows(a.offs, a.experts, a.rows, e, row0, len);
            x.k = uniform(len);
            x.i0 = bi * TM;
            left = a.wide - x.i0;
        } else {
            band_tile(t, tm, tn, bi, bj);
            find_row_tile<TM>(a, uniform(bi), e, row0, left);
            x.i0 = 0;
            x.k = MODE == kForward ? a.width : a.wide;
        }
        x.e = uniform(e);
        x.row0 = uniform(row0);
        x.left = uniform(left);
        x.c0 = uniform(bj) * TJ;
        return x;
    }
};

template <int MODE, typename TILE, bool GATED, int F>
struct LinearTask {
    static constexpr bool PT = MODE == kGradW, QT = MODE != kForward;
    typedef LinearStages<TILE, PT, QT, F> S;
    static constexpr int TM = TILE::TM, TN = TILE::TN, TJ = GATED ? TN / 2 : TN;

    // operands of a tile
    static __device__ __forceinline__ void operands(const LinearArgs &a, const TileAt &x, S &st)
    {
        // bytes of k of one row, in whole chunks: rows whose length is not are padded
        const int kb = F != kBf16 ? x.k : 2 * ((x.k + 7) & ~7);
        st.stages = MODE == kGradW ? (x.k + 63) / 64 : (kb + kRowBytes - 1) / kRowBytes;
        st.live = MODE == kGradW ? 8 : ((kb - 1) % kRowBytes + 16) / 16;
        if constexpr (MODE == kGradW) {
            st.p.set_turned(a.p + x.row0 * a.ldp + (int64_t)x.i0 * 2, a.ldp, (uint32_t)(((a.wide + 7) & ~7) - x.i0) * 2, x.k);
            st.q.set_turned(a.q + x.row0 * a.ldq + (int64_t)x.c0 * 2, a.ldq, (uint32_t)(((a.n + 7) & ~7) - x.c0) * 2, x.k);
        } else {
            const int rows = min(x.left, TM);
            st.p.set_rows(a.p + x.row0 * a.ldp, a.ldp, (uint32_t)((rows - 1) * a.ldp) + kb,
                          [&](int r) { return r < rows ? r : -1; });
            const char *q = a.q + x.e * a.qe;
            if constexpr (QT) {
                st.q.set_turned(q + (int64_t)x.c0 * 2, a.ldq, (uint32_t)(((a.n + 7) & ~7) - x.c0) * 2, a.wide);
            } else {
                // tile row r: gated, fragments of 16 rows of the gate and of
                // the value in turn
                const int n = a.n - x.c0;
                auto row = [&](int r) {
                    const int at = GATED ? (r >> 5) * 16 + (r & 15) : r;
                    return at >= n ? -1 : GATED && (r & 16) ? at + a.n : at;
                };
                const int last = GATED ? a.wide - 1 - x.c0 : min(n, TN) - 1;
                st.q.set_rows(q + x.c0 * a.ldq, a.ldq, (uint32_t)(last * a.ldq) + kb, row);
                if constexpr (F == kMxWords) {
#pragma unroll
                    for (int l = 0; l < S::LS; ++l) {
                        const int t = l * TILE::THREADS + threadIdx.x, r = row(min(max(t - TM, 0), TN - 1));
                        st.scales[l] = t < TM ? a.sp + (x.row0 + min(t, rows - 1)) * a.ldsp
                                              : a.sq + x.e * a.sqe + (int64_t)(x.c0 + max(r, 0)) * a.ldsq;
                    }
                }
                if constexpr (F == kMxBytes) {
                    // rows past the last: another one's, whose results are dropped
                    const int wave = uniform(threadIdx.x >> 6), fr = threadIdx.x & 15;
#pragma unroll
                    for (int i = 0; i < TILE::FP; ++i)
                        st.byte_p[i] = a.sp + (x.row0 + min((wave / TILE::WN * TILE::FP + i) * 16 + fr, rows - 1)) * a.ldsp;
#pragma unroll
                    for (int j = 0; j < TILE::FQ; ++j)
                        st.byte_q[j] = a.sq + x.e * a.sqe +
                                       (int64_t)(x.c0 + max(row((wave % TILE::WN * TILE::FQ + j) * 16 + fr), 0)) * a.ldsq;
                    st.stride_p = a.sbp;
                    st.stride_q = a.sbq;
                    st.blocks = x.k / 32;
                }
            }
        }
    }

    static __device__ __forceinline__ void clear(const LinearArgs &a, const TileAt &x)
    {
        clear_tile<TM, TJ, TILE::THREADS>(a.out, a.so, x.row0, x.left, x.c0, a.n);
        if (MODE == kForward && a.pre) {
            clear_tile<TM, TJ, TILE::THREADS>(a.pre, a.spre, x.row0, x.left, x.c0, a.n);
            if (GATED)
                clear_tile<TM, TJ, TILE::THREADS>(a.pre + a.n, a.spre, x.row0, x.left, x.c0, a.n);
        }
    }

    static __device__ __forceinline__ void start(float4v (&acc)[TILE::FP][TILE::FQ])
    {
#pragma unroll
        for (int i = 0; i < TILE::FP; ++i)
#pragma unroll
            for (int j = 0; j < TILE::FQ; ++j)
                acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }

    static __device__ __forceinline__ void store(const LinearArgs &a, const TileAt &x, float4v (&acc)[TILE::FP][TILE::FQ])
    {
        uint16_t *out = MODE == kGradW ? a.out + x.e * a.oe : a.out;
        linear_store<TILE, GATED, MODE == kForward>(a, acc, x.e, MODE == kGradW ? x.i0 : x.row0, x.left, x.c0, a.n, out, a.so);
    }
};

// One tile, or with SPLIT a part of its sum, per workgroup; two or three of
// those on a CU cover each other's waits.  128 rows over 50 of 64 gated experts of
// 768 x 2048 70 us: weights at 4.4 TB/s, waves waiting in 52% of their cycles.
template <int MODE, typename TILE, bool GATED, int F, bool SPLIT>
__global__ __launch_bounds__(TILE::THREADS, 2) void linear_kernel(LinearArgs a)
{
    typedef LinearTask<MODE, TILE, GATED, F> Task;
    __shared__ __attribute__((aligned(16))) char lds[TILE::NST * Task::S::BYTES];
    const LinearGrid<MODE, TILE, GATED> grid(a);
    const int work = SPLIT ? grid.total * a.splits : grid.total;
    int t = spread(blockIdx.x, work), part = 0;
    if (t >= work)
        return;
    if constexpr (SPLIT) {
        part = uniform(t / grid.total);
        t -= part * grid.total;
    }
    const TileAt x = grid.at(a, t);
    if (MODE != kGradW && x.e >= a.experts) {
        if (!SPLIT)
            Task::clear(a, x);
        return;
    }
    typename Task::S st;
    st.lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    Task::operands(a, x, st);
    if constexpr (SPLIT)
        st.part(uniform(st.stages * part / a.splits), uniform(st.stages * (part + 1) / a.splits));
    float4v acc[TILE::FP][TILE::FQ];
    Task::start(acc);
    const int wave = uniform(threadIdx.x >> 6);
    if (st.stages > 0)
        linear_pipeline<TILE, Task::PT, Task::QT, F>(st, wave / TILE::WN * TILE::FP * 16, wave % TILE::WN * TILE::FQ * 16, acc);
    if constexpr (SPLIT) {
        // grad W: experts' results one after the other
        const int64_t row0 = MODE == kGradW ? (int64_t)x.e * a.wide + x.i0 : x.row0;
        store_part<TILE, GATED>(a, acc, row0, x.left, x.c0, a.n, a.parts + part * a.part_size);
    } else {
        Task::store(a, x, acc);
    }
}

// The parts of the sums, in order, and what follows the product: a workgroup per
// result row and 1024 columns.  MODE and GATED as of the product.  A pass over
// splits x 4 bytes per sum, bound by latency: 92 rows x 3904 x 577 gated in 7
// parts 15 us a call (20 with one part's loads at a time).
template <int MODE, bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a)
{
    const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int64_t all = MODE == kGradW ? (int64_t)a.experts * a.wide : a.rows;
    for (int64_t r = blockIdx.x; r < all; r += gridDim.x) {
        int e = 0;
        uint16_t *out = a.out + r * a.so;
        bool none = false;
        if constexpr (MODE == kGradW) {
            e = uniform((int)(r / a.wide));
            out = a.out + e * a.oe + (r - (int64_t)e * a.wide) * a.so;
        } else if (a.offs) {
            // the group that holds row r: the first that ends past it
            int g0 = 0;
            for (;; g0 += 64) {
                const int g = g0 + (threadIdx.x & 63);
                const uint64_t past = __ballot(g >= a.experts || min(max(a.offs[g], 0), a.rows) > r);
                if (past) {
                    e = g0 + __builtin_ctzll(past);
                    break;
                }
            }
            none = e >= a.experts;
        }
        if (c >= a.n)
            continue;
        // four parts' loads before their sums
        auto sum = [&](int64_t at) {
            const float *from = a.parts + r * a.ldparts + at;
            float4v v = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int p = 0; p < a.splits; p += 4) {
                float4v x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    x[u] = *reinterpret_cast<const float4v *>(from + min(p + u, a.splits - 1) * a.part_size);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (p + u < a.splits)
                        v += x[u];
            }
            return v;
        };
        float4v v = {0.0f, 0.0f, 0.0f, 0.0f}, g = v;
        if (!none) {
            v = sum(c);
            if (GATED)
                g = sum(a.ldparts / 2 + c);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = c + k;
            if (at >= a.n)
                continue;
            float y = v[k];
            if constexpr (MODE == kForward) {
                const bool bias = a.bias && !none;
                y += bias ? bias_at(a.bias, a.bias_f32, e * a.sb + at) : 0.0f;
                if (a.pre)
                    a.pre[r * a.spre + at] = Piece<uint16_t>::from_f32(y);
                y = act_value(a.act, y);
                if constexpr (GATED) {
                    const float z = g[k] + (bias ? bias_at(a.bias, a.bias_f32, e * a.sb + a.n + at) : 0.0f);
                    if (a.pre)
                        a.pre[r * a.spre + a.n + at] = Piece<uint16_t>::from_f32(z);
                    y *= z;
                }
                if (a.resid && !none)
                    y += Piece<uint16_t>::to_f32(a.resid[r * a.sr + at]);
            }
            out[at] = Piece<uint16_t>::from_f32(y);
        }
    }
}

// A workgroup per CU takes one tile after the other: where the next one is and
// its first loads come before the results of the last are written, so that
// neither the search nor the first loads' latency is waited for.  In MXFP8 that
// holds in part: the registers do not suffice, the compiler spills 3 of them, of
// the gated form 14, and their reloads between two tiles wait for the loads that
// are on their way.  A last round of at most half the workgroups is taken as half
// tiles by all of them.
// Bound by the matrix units and, above 60% of their cycles, by the clock that
// their power leaves: 8192 x 5120 x 8192 with GELU 543 us, 1.27 PFLOP/s, MFMA busy
// 70% (gradients 576 and 582, 60-63%: the transposing reads take two per
// fragment); MXFP8 16384 x 5120 x 8192 746, 1.84 PFLOP/s, 45%, and no one bound
// that was found: a stage takes some 2050 cycles of scaled products at the nominal
// rate, its fragments (196 KB) 1540 of LDS reads.  On 64 x 64 tiles product and
// gradients took 3662 together (1759 here), MXFP8 1592.
template <int MODE, bool GATED, int F>
__global__ __launch_bounds__(LinearLarge::THREADS, 2) void linear_large_kernel(LinearArgs a)
{
    typedef LinearTask<MODE, LinearLarge, GATED, F> Task;
    typedef LinearTask<MODE, LinearHalf, GATED, F> Half;
    typedef LinearAlternating<LinearLarge, Task::PT, Task::QT, F> Loop;
    typedef LinearAlternating<LinearHalf, Task::PT, Task::QT, F> HalfLoop;
    __shared__ __attribute__((aligned(16))) char lds[2 * Task::S::BYTES];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const LinearGrid<MODE, LinearLarge, GATED> grid(a);
    const int wgs = gridDim.x, rest = uniform(grid.total % wgs), whole = 2 * rest <= wgs ? grid.total - rest : grid.total;
    const int padded = (whole + 255) & ~255;
    const int wave = uniform(threadIdx.x >> 6), wp = wave >> 2, wq = wave & 3;
    typename Task::S st;
    st.lds0 = lds0;
    // the next tile of this workgroup from grid number b on
    auto next = [&](int &b, TileAt &x) {
        for (; b < padded; b += wgs) {
            const int t = spread(b, whole);
            if (t >= whole)
                continue;
            x = grid.at(a, t);
            b += wgs;
            return true;
        }
        return false;
    };
    int b = blockIdx.x;
    TileAt x, y;
    bool more = next(b, x);
    auto sums = [&](const TileAt &t) { return MODE == kGradW ? t.k > 0 : t.e < a.experts && t.k > 0; };
    if (more && sums(x)) {
        Task::operands(a, x, st);
        Loop::first_loads(st);
    }
    while (more) {
        more = next(b, y);
        if (MODE != kGradW && x.e >= a.experts) {
            if (more && sums(y)) {
                Task::operands(a, y, st);
                Loop::first_loads(st);
            }
            Task::clear(a, x);
        } else {
            float4v acc[LinearLarge::FP][LinearLarge::FQ];
            Task::start(acc);
            if (sums(x))
                Loop(st, wp * 128, wq * 64).run(acc);
            if (more && sums(y)) {
                Task::operands(a, y, st);
                Loop::first_loads(st);
            }
            Task::store(a, x, acc);
        }
        x = y;
    }
    if (whole == grid.total)
        return;
    const int id = spread(blockIdx.x, 2 * rest);
    if (id >= 2 * rest)
        return;
    x = grid.at(a, whole + (id >> 1));
    x.c0 += (id & 1) * Half::TJ;
    if (x.c0 >= a.n)
        return;
    if (MODE != kGradW && x.e >= a.experts) {
        Half::clear(a, x);
        return;
    }
    typename Half::S hs;
    hs.lds0 = lds0;
    float4v acc[LinearHalf::FP][LinearHalf::FQ];
    Half::start(acc);
    if (sums(x)) {
        Half::operands(a, x, hs);
        HalfLoop::first_loads(hs);
        HalfLoop(hs, wp * 128, wq * 32).run(acc);
    }
    Half::store(a, x, acc);
}

// ---------------------------------------------------------------- few rows

// Up to 16 rows in all: bound by the weights, which go straight from memory into
// registers.  A workgroup has 16 rows of W (gated: 16 of the gate and of the
// value) of one expert against the group's rows, all of which one matrix
// instruction takes; its eight waves take the parts of the sum and meet in LDS.
// A wave asks for 256 of k at a time (MXFP8: 512) and multiplies before it asks
// again: sums over 4096, 512 a wave, are two latencies one after the other.  The
// grid has every expert, also those without a row, which end at once.  One row x
// 4096 x 4096 (34 MB of weights) 11 us a call, 16 rows x 5120 x 8192 (84 MB) 30.
constexpr int kFewWaves = 8, kFewRows = 16;

template <int NF, int U>
__device__ __forceinline__ void few_range(const LinearArgs &a, const char *const (&w)[NF], const char *x, bool there,
                                          int k0, int k1, float4v (&acc)[NF])
{
    int k = k0;
    for (; k + U * 32 <= k1; k += U * 32) {
        WeightStep<false> s[NF][U];
        bf16x8 t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
                s[i][u].load(w[i], nullptr, k + u * 32);
            t[u] = there ? token_piece<false>(reinterpret_cast<const uint16_t *>(x), k + u * 32, 0) : zero_piece();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[i][u].piece(0), t[u], acc[i], 0, 0, 0);
    }
    for (; k < k1; k += 32) {
        WeightStep<false> s[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i)
            s[i].load_tail(w[i], nullptr, k, a.width);
        const bf16x8 t = there ? token_piece_tail<false>(reinterpret_cast<const uint16_t *>(x), k, 0, a.width) : zero_piece();
#pragma unroll
        for (int i = 0; i < NF; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[i].piece(0), t, acc[i], 0, 0, 0);
    }
}

template <int NF, int U>
__device__ __forceinline__ void few_range_mx(const LinearArgs &a, const char *const (&w)[NF], const uint8_t *const (&ws)[NF],
                                             const char *x, const uint8_t *xs, bool there, int k0, int k1, float4v (&acc)[NF])
{
    auto some = [&](auto steps, int k, int end) {
        constexpr int N = decltype(steps)::value;
        int8v s[N][NF], t[N];
        int ss[N][NF], ts[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                s[u][i] = scaled_values(reinterpret_cast<const uint8_t *>(w[i]), k + u * 128, end, true);
                ss[u][i] = scaled_scale(ws[i], a.sbq, k + u * 128, end, true);
            }
            t[u] = scaled_values(reinterpret_cast<const uint8_t *>(x), k + u * 128, end, there);
            ts[u] = scaled_scale(xs, a.sbp, k + u * 128, end, there);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
                acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(s[u][i], t[u], acc[i], 0, 0, 0, ss[u][i], 0, ts[u]);
    };
    int k = k0;
    for (; k + U * 128 <= k1; k += U * 128)
        some(std::integral_constant<int, U>(), k, 1 << 30);
    for (; k < k1; k += 128)
        some(std::integral_constant<int, 1>(), k, a.width);
}

template <bool GATED, bool MX>
__global__ __launch_bounds__(kFewWaves * 64) void linear_few_kernel(LinearArgs a)
{
    constexpr int NF = GATED ? 2 : 1, STEP = MX ? 128 : 32, U = MX ? 4 : 8;
    __shared__ float4v sums[kFewWaves][NF][64];
    const int e = blockIdx.y, c0 = blockIdx.x * 16, wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, fr = lane & 15;
    int start, len;
    group_rows(a.offs, a.experts, a.rows, e, start, len);
    start = uniform(start);
    len = uniform(len);
    if (len == 0)
        return;
    if (e >= a.experts) {
        clear_tile<kFewRows, 16, kFewWaves * 64>(a.out, a.so, start, len, c0, a.n);
        if (a.pre) {
            clear_tile<kFewRows, 16, kFewWaves * 64>(a.pre, a.spre, start, len, c0, a.n);
            if (GATED)
                clear_tile<kFewRows, 16, kFewWaves * 64>(a.pre + a.n, a.spre, start, len, c0, a.n);
        }
        return;
    }
    const char *w[NF];
    const uint8_t *ws[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        // past the last row: the last one's, whose results are dropped
        const int64_t r = min(c0 + fr, a.n - 1) + i * a.n;
        w[i] = a.q + e * a.qe + r * a.ldq;
        ws[i] = MX ? a.sq + e * a.sqe + r * a.ldsq : nullptr;
    }
    const int steps = (a.width + STEP - 1) / STEP;
    const int k0 = steps * wave / kFewWaves * STEP, k1 = min(steps * (wave + 1) / kFewWaves * STEP, a.width);
    const bool there = fr < len;
    const int64_t own = start + (there ? fr : 0);
    float4v acc[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i)
        acc[i] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (MX)
        few_range_mx<NF, U>(a, w, ws, a.p + own * a.ldp, a.sp + own * a.ldsp, there, k0, k1, acc);
    else
        few_range<NF, U>(a, w, a.p + own * a.ldp, there, k0, k1, acc);
#pragma unroll
    for (int i = 0; i < NF; ++i)
        sums[wave][i][lane] = acc[i];
    __syncthreads();
    // a lane of the first wave has four columns of a row
    if (wave > 0 || !there)
        return;
    float4v z[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        z[i] = sums[0][i][lane];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v)
            z[i] += sums[v][i][lane];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = c0 + 4 * (lane >> 4) + k;
        if (c >= a.n)
            continue;
        float v = z[0][k] + (a.bias ? bias_at(a.bias, a.bias_f32, e * a.sb + c) : 0.0f);
        if (a.pre)
            a.pre[own * a.spre + c] = Piece<uint16_t>::from_f32(v);
        v = act_value(a.act, v);
        if constexpr (GATED) {
            const float g = z[1][k] + (a.bias ? bias_at(a.bias, a.bias_f32, e * a.sb + a.n + c) : 0.0f);
            if (a.pre)
                a.pre[own * a.spre + a.n + c] = Piece<uint16_t>::from_f32(g);
            v *= g;
        }
        if (a.resid)
            v += Piece<uint16_t>::to_f32(a.resid[own * a.sr + c]);
        a.out[own * a.so + c] = Piece<uint16_t>::from_f32(v);
    }
}

// ---------------------------------------------------------------- around them

// (count, rows, cols) elements of bf16 in rows padded with zeros to `padded`
// elements (a multiple of 8), for operands whose rows do not start on 16 bytes
// or whose length is no multiple of 8.  2^shift threads take a row, of all
// matrices one after the other.  Bound by memory: 38 MB read and 36 written in
// 15 us, 4.8 TB/s.
struct LinearCopy {
    const uint16_t *in;
    int64_t se, sr;
    int rows, cols, padded, shift;
    uint32_t all;                 // rows of all matrices
    int blocks;                   // workgroups
    uint16_t *out;
};

constexpr int kCopies = 3;

// all of a call's copies in one launch
struct LinearCopies {
    LinearCopy c[kCopies];
};

__global__ __launch_bounds__(256) void linear_pack_kernel(LinearCopies list)
{
    int block = blockIdx.x, n = 0;
    while (n + 1 < kCopies && block >= list.c[n].blocks)
        block -= list.c[n++].blocks;
    const LinearCopy &c = list.c[n];
    const uint32_t thread = block * 256 + threadIdx.x, step = c.blocks * 256 >> c.shift;
    const int first = (int)(thread & ((1u << c.shift) - 1)) * 8;
    for (uint32_t row = thread >> c.shift; row < c.all; row += step) {
        const uint32_t e = row / (uint32_t)c.rows, r = row - e * (uint32_t)c.rows;
        const uint16_t *src = c.in + e * c.se + r * c.sr;
        uint16_t *dst = c.out + (int64_t)row * c.padded;
        for (int k = first; k < c.padded; k += 8 << c.shift)
            st_piece<uint16_t>(dst + k, load8(src, k, c.cols));
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
// parts of SLICE rows.
//   plain  dz = dy act'(z)        gated  dz = [dy value act'(gate), dy act(gate)]
// dz is rounded to bf16, the type that the two products take; the sums are of
// the values before that rounding.  A wave has every fourth row of a slice and
// 512 columns.  `most`: slices that parts has room for, which only group ends that
// decrease exceed.  Bound by memory: 8192 x 8192 97 us, 4.2 TB/s; gated 32768 x 2048
// 167, 3.9 TB/s.
template <bool GATED, bool PRE, int ACT, int SLICE>
__global__ __launch_bounds__(256) void linear_dact_kernel(LinearArgs a, const uint16_t *__restrict__ dy, int64_t sy,
                                                          const uint16_t *__restrict__ pre, int64_t spre,
                                                          uint16_t *dz, int64_t sdz, float *parts, int most)
{
    __shared__ float sums[4][GATED ? 2 : 1][512];
    const int slices = min(count_row_tiles<SLICE>(a), most);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = GATED ? a.wide / 2 : a.wide;
    const int c = blockIdx.y * 512 + lane * 8;
    for (int s = blockIdx.x; s < slices; s += gridDim.x) {
        int e, row0, left;
        find_row_tile<SLICE>(a, s, e, row0, left);
        if (e >= a.experts)
            return;  // and so are all slices after it
        const int end = min(left, SLICE);
        float total[GATED ? 2 : 1][8] = {};
        // four rows at a time: their loads before their values
        constexpr int AT_ONCE = 4;
        for (int r0 = wave; r0 < end && c < n; r0 += 4 * AT_ONCE) {
            Piece<uint16_t> d[AT_ONCE], z[AT_ONCE], w[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int64_t row = (int64_t)row0 + min(r0 + 4 * i, end - 1);
                d[i] = load8(dy + row * sy, c, n);
                if constexpr (PRE)
                    z[i] = load8(pre + row * spre, c, n);
                if constexpr (GATED)
                    w[i] = load8(pre + row * spre + n, c, n);
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                if (r0 + 4 * i >= end)
                    continue;
                float g[8], v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    g[k] = d[i].get(k);
                if constexpr (PRE) {
                    uint16_t *to = dz + ((int64_t)row0 + r0 + 4 * i) * sdz;
                    if constexpr (GATED) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float y, slope;
                            act_both(ACT, z[i].get(k), y, slope);
                            v[k] = g[k] * y;
                            g[k] = g[k] * w[i].get(k) * slope;
                        }
                        store8(to, c, n, g);
                        store8(to + n, c, n, v);
                        if (c + 8 >= n)
                            for (int k = 2 * n; k < sdz; ++k)  // the padding
                                to[k] = 0;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float y, slope;
                            act_both(ACT, z[i].get(k), y, slope);
                            g[k] *= slope;
                        }
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

// The slices' sums of each group in fp64: a workgroup per group and 64 columns,
// every fourth slice to a wave, the waves in order.  Latency: 5 us for 4 MB.
__global__ __launch_bounds__(256) void linear_bias_kernel(LinearArgs a, int slice, const float *__restrict__ parts,
                                                          int most, float *__restrict__ out)
{
    __shared__ double sums[4][64];
    const int e = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int before = 0, own = 0, start, len;
    for (int g = lane; g <= e; g += 64) {
        group_rows(a.offs, a.experts, a.rows, g, start, len);
        const int n = (len + slice - 1) / slice;
        (g < e ? before : own) += n;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        before += __shfl_xor(before, m, 64);
        own += __shfl_xor(own, m, 64);
    }
    before = min(max(before, 0), most);
    own = min(own, most - before);
    const int c = blockIdx.x * 64 + lane;
    double s = 0.0;
    if (c < a.wide) {
        const float *p = parts + (int64_t)before * a.wide + c;
#pragma unroll 8
        for (int i = wave; i < own; i += 4)
            s += p[(int64_t)i * a.wide];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < a.wide)
        out[(int64_t)e * a.wide + c] = (float)((sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]));
}

}  // namespace mxq
