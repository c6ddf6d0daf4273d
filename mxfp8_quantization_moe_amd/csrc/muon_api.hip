// C entry points of the Newton-Schulz orthogonalisation: argument checks, the
// workspace's layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mxq.h"
#include "api_common.hpp"
#include "muon_kernels.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxDim = 65536;

// large: 128 KB of LDS, one workgroup of eight alternating waves per CU;
// medium: 72 KB, two per CU; small: 48 KB, three per CU
using TileLarge = MuonTile<256, 256, 2, 4, 64, 2>;
using TileHalf = MuonTile<256, 128, 2, 4, 64, 2>;
using TileMedium = MuonTile<128, 64, 4, 2, 64, 3>;
using TileSmall = MuonTile<64, 64, 2, 2, 64, 3>;

struct MuonPlan {
    int tile;            // 2 large, 1 medium, 0 small
    int64_t mp, np;      // padded extents, m <= n
    int64_t bytes;
};

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Larger tiles do more per loaded byte, smaller ones fill the machine from
// fewer rows and pad less.  Measured, five steps in us with small / medium /
// large tiles:
//     1 x  512 x  512   103 /  121 /  211     4 x 1024 x 1024   255 /  239 /  327
//     2 x 1024 x 1024   175 /  183 /  307     8 x  512 x 1024   164 /  158 /  254
//     1 x 2048 x 2048   425 /  367 /  484    12 x  768 x 2048   534 /  487 /  507
//     8 x 1024 x 1024   397 /  385 /  355    16 x  768 x 2048   686 /  632 /  554
//     2 x 2048 x 2048   665 /  611 /  531     1 x 4096 x 4096  2292 / 2007 / 1359
//     3 x 1000 x  777   175 /  190 /  319     4 x  987 x  872   220 /  195 /  323
// Medium tiles win from four workgroups on for five CUs (of 128 x 128); large ones
// when B X has tiles for a good third of the CUs and the symmetric products,
// which have about half as many, have enough of them for their length.  A size
// whose padding costs more than its rate gains is not taken (1.33 times medium
// over large, 1.12 small over medium).
MuonPlan muon_plan(int64_t count, int64_t rows, int64_t cols)
{
    const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
    auto up = [](int64_t v, int64_t t) { return (v + t - 1) / t; };
    auto volume = [&](int64_t tm, int64_t tn) { return (double)round_up(m, tm) * round_up(m, tm) * round_up(n, tn); };
    const int64_t tm = up(m, 256), tiles = count * tm * up(n, 256), lower = count * (tm * (tm + 1) / 2);
    MuonPlan p;
    if (tiles >= 96 && lower * m >= 65536 && volume(256, 256) <= 1.33 * volume(128, 64))
        p.tile = 2;
    else if (count * up(m, 128) * up(n, 128) >= 205 && volume(128, 64) <= 1.12 * volume(64, 64))
        p.tile = 1;
    else
        p.tile = 0;
    p.mp = round_up(m, p.tile == 2 ? 256 : p.tile == 1 ? 128 : 64);
    p.np = round_up(n, p.tile == 2 ? 256 : 64);
    p.bytes = count * (5 * p.mp * p.np + 5 * p.mp * p.mp + 8 * p.mp + 8 * kNormParts);
    return p;
}

bool sizes_ok(int64_t count, int64_t rows, int64_t cols)
{
    return count >= 0 && rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim && count <= 65535;
}

// A grid of large tiles runs in rounds of one tile per CU.  A last round of at
// most half the CUs is taken as half tiles instead, by all of them: two of 2048 x
// 2048 546 us, 730 without; eight of 2048 x 4096 2.84 ms, 2.99; one 8192 x 5120
// 3.37, 3.42.
constexpr int64_t kCUs = 256;

template <int MODE, typename TILE, typename HALF>
void launch_product(const MuonBuffers &b, const MuonStep &st, int64_t count, uint16_t *out, const MuonView &ov,
                    hipStream_t s)
{
    constexpr bool SYM = MODE == kModeA || MODE == kModeB;
    const int64_t tm = b.mp / TILE::TM, tn = b.np / TILE::TN;
    const int64_t tiles = count * (SYM ? TILE::SS * (tm * (tm + 1) / 2) : tm * tn);
    const int64_t rest = std::is_same<TILE, HALF>::value || tiles % kCUs > kCUs / 2 ? 0 : tiles % kCUs;
    muon_product_kernel<MODE, TILE, HALF><<<dim3((unsigned)(tiles + rest)), dim3(TILE::THREADS), 0, s>>>(
        b, st, out, ov, (int)(tiles - rest));
}

// X X^T of a long matrix has few tiles with long sums: each sum is then taken
// in up to 8 parts of at least 12 stages, as many as `at_once` workgroups of
// the tile run at a time and as fit where the next X will be, and joined by a
// kernel of its own.  Five steps, without / with: 1 x 64 x 8192 191 / 101 us,
// 3 x 175 x 7481 233 / 160, 1 x 256 x 4096 155 / 117, 1 x 2048 x 8192 932 /
// 871; a sum of less than 32 stages loses by the launch (17 x 126 x 1327 106 /
// 122), and so do medium tiles past one per CU (2 x 1024 x 4096 363 / 370).
template <typename TILE>
int sum_splits(const MuonBuffers &b, int64_t count, int64_t at_once)
{
    const int64_t tm = b.mp / TILE::TM, tiles = count * TILE::SS * (tm * (tm + 1) / 2), stages = b.np / TILE::BK;
    if (stages < 32)
        return 1;
    const int64_t room = b.np / (2 * b.mp);  // fp32 of mp x mp in f16 of mp x np
    return (int)std::max<int64_t>(1, std::min({(int64_t)8, at_once / tiles, stages / 12, room}));
}

template <typename TILE>
void launch_parts(const MuonBuffers &b, const MuonStep &st, int64_t count, hipStream_t s)
{
    const int64_t tm = b.mp / TILE::TM, tiles = count * TILE::SS * (tm * (tm + 1) / 2), t64 = b.mp / 64;
    const int64_t whole = count * b.mp * b.mp;
    const MuonView parts = {whole, 0, 0, 0, 0};
    muon_product_kernel<kModePart, TILE, TILE><<<dim3((unsigned)(tiles * b.splits)), dim3(TILE::THREADS), 0, s>>>(
        b, st, nullptr, parts, (int)tiles);
    muon_join_kernel<<<dim3((unsigned)(t64 * (t64 + 1) / 2), (unsigned)count), dim3(256), 0, s>>>(b, st, whole);
}

template <typename TILE, typename HALF>
void launch_steps(MuonBuffers &b, MuonStep st, int steps, int64_t count, int64_t at_once, uint16_t *out,
                  const MuonView &ov, hipStream_t s)
{
    b.splits = sum_splits<TILE>(b, count, at_once);
    for (int k = 0; k < steps; ++k) {
        if (b.splits > 1)
            launch_parts<TILE>(b, st, count, s);
        else
            launch_product<kModeA, TILE, HALF>(b, st, count, out, ov, s);
        launch_product<kModeB, TILE, HALF>(b, st, count, out, ov, s);
        if (k + 1 < steps)
            launch_product<kModeX, TILE, HALF>(b, st, count, out, ov, s);
        else
            launch_product<kModeOut, TILE, HALF>(b, st, count, out, ov, s);
        st.cur ^= 1;
    }
}

template <typename T>
void launch_load(const void *g, const MuonView &gv, MuonBuffers &b, int count, float eps, hipStream_t s)
{
    const T *p = reinterpret_cast<const T *>(g);
    // as rows along the unit stride; one row when they follow one another
    int64_t inner = gv.sj == 1 ? gv.n : gv.m, outer = gv.sj == 1 ? gv.m : gv.n;
    const int64_t so = gv.sj == 1 ? gv.si : gv.sj;
    if (so == inner) {
        inner *= outer;
        outer = 1;
    }
    const int64_t span = kNormThreads * kNormLoads * Piece<T>::N;
    b.parts = (int)std::min<int64_t>(kNormParts, outer * ((inner + span - 1) / span));
    muon_norm_kernel<T><<<dim3((unsigned)b.parts, (unsigned)count), dim3(kNormThreads), 0, s>>>(p, gv.se, inner, outer, so, b.part);
    muon_load_kernel<T><<<dim3((unsigned)(b.np / 64), (unsigned)(b.mp / 64), (unsigned)count), dim3(256), 0, s>>>(
        p, gv, b, eps);
}

}  // namespace

extern "C" {

int64_t mxq_muon_workspace_bytes(int64_t count, int64_t rows, int64_t cols)
{
    if (!sizes_ok(count, rows, cols))
        return -1;
    return count == 0 || rows == 0 || cols == 0 ? 0 : muon_plan(count, rows, cols).bytes;
}

mxq_status mxq_muon_orthogonalize(const void *g, int32_t dtype, int64_t count, int64_t rows, int64_t cols,
                                  int64_t sg_e, int64_t sg_r, int64_t sg_c, uint16_t *out, int64_t so_e,
                                  int64_t so_r, int64_t so_c, int32_t steps, float a, float b, float c, float eps,
                                  float scale, void *workspace, int64_t workspace_bytes, void *stream)
{
    if ((dtype != MXQ_BF16 && dtype != MXQ_F32) || !sizes_ok(count, rows, cols) || steps < 0 || steps > 1000 ||
        !(eps >= 0.0f))
        return MXQ_ERR_INVALID_ARG;
    if (count == 0 || rows == 0 || cols == 0)
        return MXQ_OK;
    if (!g || !out || !aligned_to(g, dtype == MXQ_BF16 ? 2 : 4) || !aligned_to(out, 2) || !aligned16(workspace))
        return MXQ_ERR_INVALID_ARG;
    if ((cols > 1 && sg_c != 1 && !(sg_r == 1 || rows == 1)) || (cols > 1 && so_c != 1 && !(so_r == 1 || rows == 1)))
        return MXQ_ERR_UNSUPPORTED;
    const MuonPlan p = muon_plan(count, rows, cols);
    if (workspace_bytes < p.bytes || !workspace)
        return MXQ_ERR_WORKSPACE;
    if (count * (p.mp / 64) * (p.np / 64) > INT32_MAX)
        return MXQ_ERR_INVALID_ARG;

    MuonBuffers buf;
    buf.mp = (int)p.mp;
    buf.np = (int)p.np;
    buf.part = reinterpret_cast<double *>(workspace);
    const int64_t nx = count * p.mp * p.np, na = count * p.mp * p.mp;
    buf.xh[0] = reinterpret_cast<_Float16 *>(buf.part + count * kNormParts);
    buf.xh[1] = buf.xh[0] + nx;
    buf.oh = buf.xh[1] + nx;
    buf.bo = buf.oh + na;
    buf.d = reinterpret_cast<float *>(buf.bo + na);
    buf.db = buf.d + count * p.mp;
    buf.xl = reinterpret_cast<uint8_t *>(buf.db + count * p.mp);
    buf.ol = buf.xl + nx;

    // X is G, or G transposed when G is tall
    const bool tall = rows > cols;
    const MuonView gv = {sg_e, tall ? sg_c : sg_r, tall ? sg_r : sg_c, (int)std::min(rows, cols),
                         (int)std::max(rows, cols)};
    const MuonView ov = {so_e, tall ? so_c : so_r, tall ? so_r : so_c, gv.m, gv.n};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dtype == MXQ_BF16)
        launch_load<uint16_t>(g, gv, buf, (int)count, eps, s);
    else
        launch_load<float>(g, gv, buf, (int)count, eps, s);
    const MuonStep st = {a, b, c, scale / kScaleX, 0};
    if (steps == 0)
        muon_copy_kernel<<<dim3((unsigned)gv.m, (unsigned)((gv.n + 255) / 256), (unsigned)count), dim3(256), 0, s>>>(
            buf, st.out_scale, out, ov);
    else if (p.tile == 2)
        launch_steps<TileLarge, TileHalf>(buf, st, steps, count, kCUs, out, ov, s);
    else if (p.tile == 1)
        launch_steps<TileMedium, TileMedium>(buf, st, steps, count, kCUs, out, ov, s);
    else
        launch_steps<TileSmall, TileSmall>(buf, st, steps, count, 3 * kCUs, out, ov, s);
    return launch_status();
}

}  // extern "C"
