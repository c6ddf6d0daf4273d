// C entry points of the experts' products: argument checks, operands whose
// rows the kernels cannot read in place, the choice of a tile and the launches.
// No allocation, no synchronisation, no read-back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mxq.h"
#include "api_common.hpp"
#include "linear_kernels.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxDim = 65536;

// 48 KB of LDS, three workgroups of four waves per CU; 72 KB, two of eight waves
using TileSmall = LinearTile<64, 64, 2, 2, 3>;
using TileMedium = LinearTile<64, 128, 2, 4, 3>;

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

bool sizes_ok(int64_t rows, int64_t width, int32_t experts, int64_t wide)
{
    return rows >= 0 && rows <= INT32_MAX - 4096 && width >= 0 && width <= kMaxDim && experts >= 1 &&
           experts <= MXQ_MAX_GROUPS && wide >= 0 && wide <= kMaxDim;
}

bool act_ok(int32_t activation, int32_t gated, int64_t wide)
{
    return activation >= MXQ_ACT_NONE && activation <= MXQ_ACT_SILU && (gated == 0 || gated == 1) &&
           (!gated || wide % 2 == 0);
}

// A bf16 operand (count, rows, cols) with unit stride along cols that the
// kernels read in place: 16-byte pieces throughout, rows that do not overlap,
// and offsets within a tile that fit 31 bits.
struct Rows {
    const void *p;
    int64_t se, sr, rows, cols;
    bool direct() const
    {
        return cols % 8 == 0 && aligned16(p) && se % 8 == 0 && sr % 8 == 0 && sr < (1 << 21) && sr >= cols;
    }
    int64_t packed_bytes(int64_t count) const { return round_up(count * rows * round_up(cols, 8) * 2, 256); }
};

// A single row's stride says nothing (0 of an expanded one), but the descriptor of
// a turned operand ends with its last row only if the rows that a stage would have
// after it lie further on.
Rows rows_of(const void *p, int64_t se, int64_t sr, int64_t rows, int64_t cols)
{
    return {p, se, rows > 1 ? sr : round_up(cols, 8), rows, cols};
}

// What a call's workspace has been used for so far.
struct Room {
    char *at, *end;
    void *take(int64_t bytes)
    {
        char *p = at;
        at += bytes;
        return p;
    }
};

// The copies that a call needs, launched together.
struct Copies {
    LinearCopies list = {};
    int n = 0, blocks = 0;
    void launch(hipStream_t st) const
    {
        if (blocks > 0)
            linear_pack_kernel<<<dim3((unsigned)blocks), dim3(256), 0, st>>>(list);
    }
};

// the operand in place or a copy in padded rows, which copies.launch() makes
Rows readable(const Rows &r, int64_t count, Room &room, Copies &copies)
{
    if (r.direct())
        return r;
    Rows to = {nullptr, 0, round_up(r.cols, 8), r.rows, r.cols};
    to.se = r.rows * to.sr;
    to.p = room.take(r.packed_bytes(count));
    const int64_t all = count * r.rows;
    if (all * to.sr > 0) {
        int shift = 0;
        while (shift < 8 && (8 << shift) < to.sr)
            ++shift;
        const int blocks = (int)std::min<int64_t>(((all << shift) + 255) / 256, 8192);
        copies.list.c[copies.n++] = {reinterpret_cast<const uint16_t *>(r.p), r.se, r.sr, (int)r.rows, (int)r.cols,
                                     (int)to.sr, shift, (uint32_t)all, blocks,
                                     const_cast<uint16_t *>(reinterpret_cast<const uint16_t *>(to.p))};
        copies.blocks += blocks;
    }
    return to;
}

// e8m0 scales (count, rows, blocks), read in words of four blocks
struct Scales {
    const uint8_t *p;
    int64_t se, sr, sb, rows, blocks;
    bool direct() const
    {
        return blocks % 4 == 0 && sb == 1 && aligned_to(p, 4) && se % 4 == 0 && sr % 4 == 0;
    }
    int64_t packed_bytes(int64_t count) const { return round_up(count * rows * round_up(blocks, 4), 256); }
};

// Grid of a copy of `items` per group, 256 a workgroup and no more than cover the
// chip: 2^28 threads at most, whatever the groups.
dim3 copy_grid(int64_t items, int64_t count)
{
    return dim3((unsigned)std::min((items + 255) / 256, std::max<int64_t>(std::min<int64_t>(8192, (1 << 20) / count), 1)), (unsigned)count);
}

Scales readable(const Scales &s, int64_t count, Room &room, hipStream_t st)
{
    if (s.direct())
        return s;
    Scales to = {nullptr, 0, round_up(s.blocks, 4), 1, s.rows, s.blocks};
    to.se = s.rows * to.sr;
    to.p = reinterpret_cast<uint8_t *>(room.take(s.packed_bytes(count)));
    const int64_t words = s.rows * to.sr / 4;
    if (words > 0)
        linear_pack_scales_kernel<<<copy_grid(words, count), dim3(256), 0, st>>>(
            s.p, s.se, s.sr, s.sb, (int)s.rows, (int)s.blocks, const_cast<uint8_t *>(to.p), (int)to.sr);
    return to;
}

// Row tiles that any group ends can need; one group has none behind it.
int64_t row_tiles(int64_t rows, int32_t experts, bool grouped, int64_t tm)
{
    const int64_t even = (rows + tm - 1) / tm;
    return grouped ? std::min<int64_t>(even + experts, rows) : even;
}

// Row tiles that groups of about equal length have.
int64_t usual_row_tiles(int64_t rows, int32_t experts, int64_t tm)
{
    if (experts == 1)
        return (rows + tm - 1) / tm;
    return 2 * rows >= experts * tm ? rows / tm + experts / 2 : std::min<int64_t>(experts, rows);
}

constexpr int64_t kCUs = 256;

enum Kernel { kFew, kSmall, kMedium, kLarge };

struct Choice {
    Kernel kernel;
    int splits;
};

// What a product runs on, by its extents alone (cols: result columns, of a gate
// and its value both).  us per call, weights out of the caches for few rows:
//   few    up to 16 rows in all: 1 row x 4096 x 4096 12.6 (27 on small tiles), 16
//          rows x 5120 x 8192 30 (34); 32 rows 43 (35)
//   large  from 72 large tiles on, that groups fill to a quarter: 4096 rows x
//          4096 x 4096 100 (medium 164, small 197), over 8 experts 159 (212, 253);
//          1024 rows over 8 experts 71 (81, 94), in one group (64 tiles) 61 (45, 56);
//          1024 rows over 64 experts of 2048 x 768 42 (41, 33); grad x of 4096
//          rows over 8 experts of 2048 x 1024 (80 tiles) 36 (48, 45)
//   medium more small tiles than the CUs hold at a time, which groups fill: 4096
//          rows over 64 experts of 1024 x 2048 56 (small 67), 1024 rows x 4096 x
//          4096 45 (56); 128 rows over 64 gated experts of 2048 x 768 79 (70).
//          grad x also of small groups: 256 rows over 64 experts of 1024 x 2048 41
//          (54).  With MXFP8 operands even or slower (1024 x 4096 x 4096 42
//          against 45, 4096 rows over 64 experts of 2048 x 768 37 against 32)
//   parts  sums of 16 stages and more with small tiles for half the room or less
// Not measured on both sides: those limits of the parts, a weight gradient of few
// stages on large tiles, and how the last round of tiles ends, which the rules do
// not look at.
Choice choose(LinearMode mode, bool mx, int64_t rows, int32_t experts, int64_t width, int64_t wide)
{
    const int64_t cols = mode == kForward ? wide : width;
    auto tiles = [&](int64_t tm, int64_t tn) {
        const int64_t r = mode == kGradW ? experts * ((wide + tm - 1) / tm) : usual_row_tiles(rows, experts, tm);
        return r * ((cols + tn - 1) / tn);
    };
    // 16 columns of an expert a workgroup: past 2^32 threads the tiles take it
    if (mode == kForward && rows <= kFewRows && (wide + 15) / 16 * (experts + 1) < ((int64_t)1 << 32) / (kFewWaves * 64))
        return {kFew, 1};
    if (tiles(256, 256) >= 72 && (mode == kGradW || rows >= 64 * (int64_t)experts))
        return {kLarge, 1};
    const int64_t small = tiles(64, 64), room = 3 * kCUs;
    const int64_t stages = mode == kGradW ? rows / experts / 64 : (mode == kForward ? width : wide) / (mx ? 128 : 64);
    if (2 * small <= room && stages >= 16 && small > 0)
        return {kSmall, (int)std::min<int64_t>({(int64_t)16, room / small, stages / 8})};
    const bool medium = !mx && small > room && (mode != kForward || rows >= 64 * (int64_t)experts);
    return {medium ? kMedium : kSmall, 1};
}

// Parts of a product's sums in the workspace: (splits, result rows, columns).
int64_t parts_bytes(LinearMode mode, int splits, int64_t rows, int32_t experts, int64_t width, int64_t wide)
{
    if (splits <= 1)
        return 0;
    const int64_t r = mode == kGradW ? experts * wide : rows, c = mode == kForward ? wide : width;
    return round_up(splits * r * round_up(c, 8) * 4, 256);
}

// a grid that `spread` covers, or 0 if it is past what one launch takes
int64_t grid_of(int64_t tiles, int64_t threads)
{
    const int64_t g = round_up(tiles, 256);
    return g * threads < ((int64_t)1 << 32) && g <= INT32_MAX ? g : 0;
}

template <int MODE, typename TILE, bool GATED, int F, bool SPLIT>
mxq_status launch_tile(const LinearArgs &a, hipStream_t st)
{
    const int64_t tj = GATED ? TILE::TN / 2 : TILE::TN, tn = (a.n + tj - 1) / tj;
    const int64_t tm = MODE == kGradW ? (int64_t)a.experts * ((a.wide + TILE::TM - 1) / TILE::TM)
                                      : row_tiles(a.rows, a.experts, a.offs != nullptr, TILE::TM);
    const int64_t grid = grid_of(tm * tn * (SPLIT ? a.splits : 1), TILE::THREADS);
    if (grid == 0)
        return MXQ_ERR_UNSUPPORTED;
    linear_kernel<MODE, TILE, GATED, F, SPLIT><<<dim3((unsigned)grid), dim3(TILE::THREADS), 0, st>>>(a);
    return launch_status();
}

template <bool GATED, bool MX>
mxq_status launch_few(const LinearArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)(a.experts + (a.offs ? 1 : 0)));
    linear_few_kernel<GATED, MX><<<grid, dim3(kFewWaves * 64), 0, st>>>(a);
    return launch_status();
}

// `room`: where parts may go
template <int MODE, bool GATED, int F>
mxq_status launch(LinearArgs a, const Choice &c, Room &room, hipStream_t st)
{
    if (a.n == 0 || (MODE == kGradW ? a.wide : a.rows) == 0)
        return MXQ_OK;
    if constexpr (F != kMxBytes) {
        if (c.kernel == kLarge) {
            const int64_t tn = (a.n + 127) / 128;
            const int64_t tm = MODE == kGradW ? a.experts * ((a.wide + 255) / 256) : row_tiles(a.rows, a.experts, a.offs != nullptr, 256);
            if (tm * tn > (1 << 30))
                return MXQ_ERR_UNSUPPORTED;
            linear_large_kernel<MODE, GATED, F><<<dim3((unsigned)kCUs), dim3(LinearLarge::THREADS), 0, st>>>(a);
            return launch_status();
        }
    }
    if constexpr (MODE == kForward)
        if (c.kernel == kFew)
            return launch_few<GATED, F != kBf16>(a, st);
    if constexpr (F == kBf16)
        if (c.kernel == kMedium)
            return launch_tile<MODE, TileMedium, GATED, F, false>(a, st);
    if (c.splits == 1)
        return launch_tile<MODE, TileSmall, GATED, F, false>(a, st);
    const int64_t rows = MODE == kGradW ? (int64_t)a.experts * a.wide : a.rows;
    a.splits = c.splits;
    a.ldparts = round_up(MODE == kForward ? a.wide : a.width, 8);
    a.part_size = rows * a.ldparts;
    a.parts = reinterpret_cast<float *>(room.take(parts_bytes((LinearMode)MODE, c.splits, a.rows, a.experts, a.width, a.wide)));
    const mxq_status s = launch_tile<MODE, TileSmall, GATED, F, true>(a, st);
    if (s != MXQ_OK)
        return s;
    linear_join_kernel<MODE, GATED><<<dim3((unsigned)std::min<int64_t>(rows, 1 << 20), (unsigned)((a.n + 1023) / 1024)), dim3(256), 0, st>>>(a);
    return launch_status();
}

template <int F>
mxq_status launch_forward(const LinearArgs &a, int gated, const Choice &c, Room &room, hipStream_t st)
{
    return gated ? launch<kForward, true, F>(a, c, room, st) : launch<kForward, false, F>(a, c, room, st);
}

// a 2-D operand or result of bf16: rows of unit stride
bool rows_ok(const void *p, int64_t n, int64_t stride, bool writes, int64_t cols)
{
    return (n == 0 || cols == 0 || p) && aligned_to(p, 2) && stride >= 0 && (!writes || n <= 1 || stride >= cols);
}

bool bias_ok(const void *bias, int32_t dtype, int64_t sb_e)
{
    return !bias || ((dtype == MXQ_BF16 || dtype == MXQ_F32) && aligned_to(bias, dtype == MXQ_BF16 ? 2 : 4) && sb_e >= 0);
}

// Offsets within a tile fit 31 bits: of a gated product its rows of W lie `wide` / 2
// apart, of others they are neighbours, which the strides' limits keep in reach.
bool reach_ok(int32_t gated, int64_t wide, int64_t stride_bytes, int64_t row_bytes)
{
    return !gated || (wide - 1) * stride_bytes + row_bytes < ((int64_t)1 << 31);
}

}  // namespace

extern "C" {

int64_t mxq_moe_linear_workspace_bytes(int64_t rows, int64_t width, int32_t num_experts, int64_t wide, int32_t aligned)
{
    if (!sizes_ok(rows, width, num_experts, wide))
        return -1;
    const Choice c = choose(kForward, false, rows, num_experts, width, wide);
    const int64_t parts = parts_bytes(kForward, c.splits, rows, num_experts, width, wide);
    if (c.kernel == kFew || (aligned && width % 8 == 0))
        return parts;
    return parts + Rows{nullptr, 0, 0, rows, width}.packed_bytes(1) + Rows{nullptr, 0, 0, wide, width}.packed_bytes(num_experts);
}

mxq_status mxq_moe_linear(const uint16_t *x, int64_t rows, int64_t width, int64_t sx_r, int64_t sx_c, const uint16_t *w,
                          int32_t num_experts, int64_t wide, int64_t sw_e, int64_t sw_n, int64_t sw_k,
                          const int32_t *offs, const void *bias, int32_t bias_dtype, int64_t sb_e, int32_t activation,
                          int32_t gated, const uint16_t *residual, int64_t sr_r, int64_t sr_c, uint16_t *y, int64_t sy_r,
                          int64_t sy_c, uint16_t *pre, int64_t sp_r, int64_t sp_c, void *workspace,
                          int64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(rows, width, num_experts, wide) || !act_ok(activation, gated, wide) || (!offs && num_experts != 1) ||
        !bias_ok(bias, bias_dtype, sb_e) || !aligned16(workspace))
        return MXQ_ERR_INVALID_ARG;
    const int64_t n = gated ? wide / 2 : wide;
    if ((width > 1 && (sx_c != 1 || sw_k != 1)) || (n > 1 && (sy_c != 1 || (residual && sr_c != 1) || (pre && sp_c != 1))))
        return MXQ_ERR_UNSUPPORTED;
    if (!rows_ok(x, rows, sx_r, false, width) || !rows_ok(w, num_experts * wide, sw_n, false, width) || sw_e < 0 ||
        !rows_ok(y, rows, sy_r, true, n) || (residual && !rows_ok(residual, rows, sr_r, false, n)) ||
        (pre && !rows_ok(pre, rows, sp_r, true, wide)))
        return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || n == 0)
        return MXQ_OK;
    const Rows xr = rows_of(x, 0, sx_r, rows, width), wr = rows_of(w, sw_e, sw_n, wide, width);
    const Choice choice = choose(kForward, false, rows, num_experts, width, wide);
    const bool few = choice.kernel == kFew;
    const int64_t need = (few || xr.direct() ? 0 : xr.packed_bytes(1)) + (few || wr.direct() ? 0 : wr.packed_bytes(num_experts)) +
                         parts_bytes(kForward, choice.splits, rows, num_experts, width, wide);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return MXQ_ERR_WORKSPACE;
    const int64_t row_bytes = round_up(width, 8) * 2;
    if (!few && !reach_ok(gated, wide, wr.direct() ? wr.sr * 2 : row_bytes, row_bytes))
        return MXQ_ERR_UNSUPPORTED;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    Room room = {reinterpret_cast<char *>(workspace), nullptr};
    Copies copies;
    const Rows xo = few ? xr : readable(xr, 1, room, copies), wo = few ? wr : readable(wr, num_experts, room, copies);
    copies.launch(st);
    LinearArgs a = {};
    a.p = reinterpret_cast<const char *>(xo.p);
    a.ldp = xo.sr * 2;
    a.q = reinterpret_cast<const char *>(wo.p);
    a.ldq = wo.sr * 2;
    a.qe = wo.se * 2;
    a.offs = offs;
    a.experts = num_experts;
    a.rows = (int)rows;
    a.width = (int)width;
    a.wide = (int)wide;
    a.n = (int)n;
    a.bias = bias;
    a.sb = sb_e;
    a.bias_f32 = bias_dtype == MXQ_F32;
    a.act = activation;
    a.resid = residual;
    a.sr = sr_r;
    a.out = y;
    a.so = sy_r;
    a.pre = pre;
    a.spre = sp_r;
    return launch_forward<kBf16>(a, gated, choice, room, st);
}

int64_t mxq_moe_linear_mx_workspace_bytes(int64_t rows, int64_t width, int32_t num_experts, int64_t wide, int32_t aligned)
{
    if (!sizes_ok(rows, width, num_experts, wide) || width % 32)
        return -1;
    const Choice c = choose(kForward, true, rows, num_experts, width, wide);
    const int64_t parts = parts_bytes(kForward, c.splits, rows, num_experts, width, wide);
    if (c.kernel != kLarge || (aligned && width % 128 == 0))
        return parts;
    return parts + Scales{nullptr, 0, 0, 1, rows, width / 32}.packed_bytes(1) +
           Scales{nullptr, 0, 0, 1, wide, width / 32}.packed_bytes(num_experts);
}

mxq_status mxq_moe_linear_mx(const uint8_t *x, int64_t rows, int64_t width, int64_t sx_r, int64_t sx_c,
                             const uint8_t *x_scales, int64_t sxs_r, int64_t sxs_b, const uint8_t *w,
                             int32_t num_experts, int64_t wide, int64_t sw_e, int64_t sw_n, int64_t sw_k,
                             const uint8_t *w_scales, int64_t sws_e, int64_t sws_n, int64_t sws_b, const int32_t *offs,
                             const void *bias, int32_t bias_dtype, int64_t sb_e, int32_t activation, int32_t gated,
                             const uint16_t *residual, int64_t sr_r, int64_t sr_c, uint16_t *y, int64_t sy_r,
                             int64_t sy_c, uint16_t *pre, int64_t sp_r, int64_t sp_c, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(rows, width, num_experts, wide) || width % 32 || !act_ok(activation, gated, wide) ||
        (!offs && num_experts != 1) || !bias_ok(bias, bias_dtype, sb_e) || !aligned16(workspace))
        return MXQ_ERR_INVALID_ARG;
    const int64_t n = gated ? wide / 2 : wide;
    if ((width > 1 && (sx_c != 1 || sw_k != 1)) || (n > 1 && (sy_c != 1 || (residual && sr_c != 1) || (pre && sp_c != 1))))
        return MXQ_ERR_UNSUPPORTED;
    if (rows > 0 && wide > 0 && width > 0 && (!x || !w || !x_scales || !w_scales))
        return MXQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || sx_r % 16 || sw_e % 16 || sw_n % 16 || sx_r < 0 || sw_e < 0 || sw_n < 0 ||
        sx_r >= (1 << 22) || sw_n >= (1 << 22) || sxs_r < 0 || sxs_b < 0 || sws_e < 0 || sws_n < 0 || sws_b < 0 ||
        !rows_ok(y, rows, sy_r, true, n) || (residual && !rows_ok(residual, rows, sr_r, false, n)) ||
        (pre && !rows_ok(pre, rows, sp_r, true, wide)))
        return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || n == 0)
        return MXQ_OK;
    const Scales xs = {x_scales, 0, sxs_r, sxs_b, rows, width / 32};
    const Scales ws = {w_scales, sws_e, sws_n, sws_b, wide, width / 32};
    const Choice choice = choose(kForward, true, rows, num_experts, width, wide);
    const bool few = choice.kernel == kFew;
    const bool words = choice.kernel == kLarge;  // else scales are read from where they are
    const int64_t need = (words && !xs.direct() ? xs.packed_bytes(1) : 0) + (words && !ws.direct() ? ws.packed_bytes(num_experts) : 0) +
                         parts_bytes(kForward, choice.splits, rows, num_experts, width, wide);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return MXQ_ERR_WORKSPACE;
    if (!few && !reach_ok(gated, wide, sw_n, width))
        return MXQ_ERR_UNSUPPORTED;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    Room room = {reinterpret_cast<char *>(workspace), nullptr};
    const Scales xo = words ? readable(xs, 1, room, st) : xs, wo = words ? readable(ws, num_experts, room, st) : ws;
    LinearArgs a = {};
    a.p = reinterpret_cast<const char *>(x);
    a.ldp = sx_r;
    a.q = reinterpret_cast<const char *>(w);
    a.ldq = sw_n;
    a.qe = sw_e;
    a.sp = xo.p;
    a.ldsp = xo.sr;
    a.sq = wo.p;
    a.ldsq = wo.sr;
    a.sqe = wo.se;
    a.sbp = xo.sb;
    a.sbq = wo.sb;
    a.offs = offs;
    a.experts = num_experts;
    a.rows = (int)rows;
    a.width = (int)width;
    a.wide = (int)wide;
    a.n = (int)n;
    a.bias = bias;
    a.sb = sb_e;
    a.bias_f32 = bias_dtype == MXQ_F32;
    a.act = activation;
    a.resid = residual;
    a.sr = sr_r;
    a.out = y;
    a.so = sy_r;
    a.pre = pre;
    a.spre = sp_r;
    return choice.kernel == kLarge || (xo.direct() && wo.direct()) ? launch_forward<kMxWords>(a, gated, choice, room, st)
                                                                   : launch_forward<kMxBytes>(a, gated, choice, room, st);
}

namespace {

// Rows of a slice of the activation's gradient: 64, or 16 where that leaves less
// than four workgroups per CU (6147 x 777 over 13 experts 25 us with 64).
int slice_rows(int64_t rows, int32_t experts, int64_t n)
{
    return usual_row_tiles(rows, experts, 64) * ((n + 511) / 512) < 4 * kCUs ? 16 : 64;
}

// Slices of all groups at most, if their ends do not decrease; the kernels take no more.
int64_t most_slices(int64_t rows, int32_t experts, int64_t n)
{
    return row_tiles(rows, experts, true, slice_rows(rows, experts, n));
}

int64_t slices_bytes(int64_t rows, int32_t experts, int64_t wide, int64_t n)
{
    return round_up(most_slices(rows, experts, n) * wide * 4, 256);
}

}  // namespace

int64_t mxq_moe_linear_backward_workspace_bytes(int64_t rows, int64_t width, int32_t num_experts, int64_t wide,
                                                int32_t activation, int32_t gated, int32_t bias, int32_t aligned)
{
    if (!sizes_ok(rows, width, num_experts, wide) || !act_ok(activation, gated, wide))
        return -1;
    const Rows z = {nullptr, 0, 0, rows, wide}, x = {nullptr, 0, 0, rows, width}, w = {nullptr, 0, 0, wide, width};
    int64_t need = bias ? slices_bytes(rows, num_experts, wide, gated ? wide / 2 : wide) : 0;
    if (activation != MXQ_ACT_NONE || gated || !aligned || wide % 8)
        need += z.packed_bytes(1);
    if (!aligned || width % 8)
        need += x.packed_bytes(1) + w.packed_bytes(num_experts);
    for (LinearMode mode : {kGradX, kGradW})
        need += parts_bytes(mode, choose(mode, false, rows, num_experts, width, wide).splits, rows, num_experts, width, wide);
    return need;
}

mxq_status mxq_moe_linear_backward(const uint16_t *grad_y, int64_t sg_r, int64_t sg_c, const uint16_t *x, int64_t rows,
                                   int64_t width, int64_t sx_r, int64_t sx_c, const uint16_t *w, int32_t num_experts,
                                   int64_t wide, int64_t sw_e, int64_t sw_n, int64_t sw_k, const int32_t *offs,
                                   const uint16_t *pre, int64_t sp_r, int64_t sp_c, int32_t activation, int32_t gated,
                                   uint16_t *grad_x, int64_t sdx_r, int64_t sdx_c, uint16_t *grad_w, int64_t sdw_e,
                                   int64_t sdw_n, int64_t sdw_k, float *grad_bias, void *workspace,
                                   int64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(rows, width, num_experts, wide) || !act_ok(activation, gated, wide) || (!offs && num_experts != 1) ||
        !aligned16(workspace) || !aligned_to(grad_bias, 4))
        return MXQ_ERR_INVALID_ARG;
    const int64_t n = gated ? wide / 2 : wide;
    const bool saved = activation != MXQ_ACT_NONE || gated;
    if ((n > 1 && (sg_c != 1 || (saved && sp_c != 1))) ||
        (width > 1 && ((grad_w && (sx_c != 1 || sdw_k != 1)) || (grad_x && (sw_k != 1 || sdx_c != 1)))))
        return MXQ_ERR_UNSUPPORTED;
    if (!rows_ok(grad_y, rows, sg_r, false, n) || (saved && !rows_ok(pre, rows, sp_r, false, wide)) ||
        (grad_w && (!rows_ok(x, rows, sx_r, false, width) || !rows_ok(grad_w, wide, sdw_n, true, width) || sdw_e < 0 ||
                    (num_experts > 1 && sdw_e < wide * sdw_n))) ||
        (grad_x && (!rows_ok(w, num_experts * wide, sw_n, false, width) || sw_e < 0 ||
                    !rows_ok(grad_x, rows, sdx_r, true, width))))
        return MXQ_ERR_INVALID_ARG;
    const Rows yr = rows_of(grad_y, 0, sg_r, rows, n), zr = {nullptr, 0, 0, rows, wide},
               xr = rows_of(x, 0, sx_r, rows, width), wr = rows_of(w, sw_e, sw_n, wide, width);
    int64_t need = grad_bias ? slices_bytes(rows, num_experts, wide, n) : 0;
    if (saved || !yr.direct())
        need += zr.packed_bytes(1);
    if (grad_w && !xr.direct())
        need += xr.packed_bytes(1);
    if (grad_x && !wr.direct())
        need += wr.packed_bytes(num_experts);
    const Choice cx = choose(kGradX, false, rows, num_experts, width, wide), cw = choose(kGradW, false, rows, num_experts, width, wide);
    if (grad_x)
        need += parts_bytes(kGradX, cx.splits, rows, num_experts, width, wide);
    if (grad_w)
        need += parts_bytes(kGradW, cw.splits, rows, num_experts, width, wide);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return MXQ_ERR_WORKSPACE;
    if (wide == 0 && !(grad_x && rows > 0))
        return MXQ_OK;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    Room room = {reinterpret_cast<char *>(workspace), nullptr};
    LinearArgs a = {};
    a.offs = offs;
    a.experts = num_experts;
    a.rows = (int)rows;
    a.width = (int)width;
    a.wide = (int)wide;
    a.act = activation;
    float *parts = grad_bias ? reinterpret_cast<float *>(room.take(slices_bytes(rows, num_experts, wide, n))) : nullptr;
    const int slice = slice_rows(rows, num_experts, n), most = (int)most_slices(rows, num_experts, n);
    Copies copies;
    Rows z = yr;
    if (saved) {
        z = {room.take(zr.packed_bytes(1)), 0, round_up(wide, 8), rows, wide};
    } else {
        z = readable(yr, 1, room, copies);
    }
    const Rows wo = grad_x ? readable(wr, num_experts, room, copies) : wr, xo = grad_w ? readable(xr, 1, room, copies) : xr;
    copies.launch(st);
    if (rows > 0 && wide > 0 && (saved || parts)) {
        const int64_t slices = row_tiles(rows, num_experts, offs != nullptr, slice);
        const dim3 grid((unsigned)std::min<int64_t>(slices, 1 << 20), (unsigned)((n + 511) / 512));
        uint16_t *dz = const_cast<uint16_t *>(reinterpret_cast<const uint16_t *>(z.p));
        auto go = [&](auto kernel) {
            kernel<<<grid, dim3(256), 0, st>>>(a, grad_y, sg_r, pre, sp_r, saved ? dz : nullptr, z.sr, parts, most);
        };
        auto by_act = [&](auto g, auto sl) {
            constexpr bool G = decltype(g)::value;
            constexpr int S = decltype(sl)::value;
            switch (activation) {
            case MXQ_ACT_RELU: go(linear_dact_kernel<G, true, kActRelu, S>); break;
            case MXQ_ACT_GELU: go(linear_dact_kernel<G, true, kActGelu, S>); break;
            case MXQ_ACT_SILU: go(linear_dact_kernel<G, true, kActSilu, S>); break;
            default: go(linear_dact_kernel<G, G, kActNone, S>); break;
            }
        };
        auto by_slice = [&](auto g) {
            slice == 16 ? by_act(g, std::integral_constant<int, 16>()) : by_act(g, std::integral_constant<int, 64>());
        };
        gated ? by_slice(std::true_type()) : by_slice(std::false_type());
    }
    if (grad_bias && wide > 0)
        linear_bias_kernel<<<dim3((unsigned)((wide + 63) / 64), (unsigned)num_experts), dim3(256), 0, st>>>(a, slice, parts, most, grad_bias);
    a.p = reinterpret_cast<const char *>(z.p);
    a.ldp = z.sr * 2;
    a.n = (int)width;
    mxq_status status = launch_status();
    if (grad_x && status == MXQ_OK && rows > 0 && width > 0) {
        LinearArgs b = a;
        b.q = reinterpret_cast<const char *>(wo.p);
        b.ldq = wo.sr * 2;
        b.qe = wo.se * 2;
        b.out = grad_x;
        b.so = sdx_r;
        status = launch<kGradX, false, kBf16>(b, cx, room, st);
    }
    if (grad_w && status == MXQ_OK && wide > 0 && width > 0) {
        LinearArgs b = a;
        b.q = reinterpret_cast<const char *>(xo.p);
        b.ldq = xo.sr * 2;
        b.out = grad_w;
        b.so = sdw_n;
        b.oe = sdw_e;
        status = launch<kGradW, false, kBf16>(b, cw, room, st);
    }
    return status;
}

}  // extern "C"
