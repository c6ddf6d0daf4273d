// C entry points of the Newton-Schulz orthogonalisation: argument checks, the
// workspace's layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mxq.h"
#include "api_common.hpp"
#include "muon_kernels.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxDim = 65536;

struct MuonPlan {
    int tile;            // tile edge of the products
    int64_t mp, np;      // padded extents, m <= n
    int64_t bytes;
};

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// 256-wide tiles reuse each operand byte most and are taken when they still
// fill the machine; smaller problems take smaller tiles.
MuonPlan muon_plan(int64_t count, int64_t rows, int64_t cols)
{
    const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
    MuonPlan p;
    auto tiles = [&](int64_t t) { return count * ((m + t - 1) / t) * ((n + t - 1) / t); };
    p.tile = tiles(256) >= 256 ? 256 : tiles(128) >= 256 ? 128 : 64;
    p.mp = round_up(m, p.tile);
    p.np = round_up(n, p.tile);
    p.bytes = count * (8 * p.mp * p.np + 6 * p.mp * p.mp + 8 * p.mp + 8 * kNormParts);
    return p;
}

bool sizes_ok(int64_t count, int64_t rows, int64_t cols)
{
    return count >= 0 && rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim && count <= 65535;
}

template <int MODE, int T>
void launch_product(const MuonBuffers &b, const MuonStep &st, int count, uint16_t *out, const MuonView &ov,
                    hipStream_t s)
{
    constexpr bool SYM = MODE == kModeA || MODE == kModeB;
    const int64_t tm = b.mp / T, tn = b.np / T;
    const int64_t blocks = count * (SYM ? tm * (tm + 1) / 2 : tm * tn);
    constexpr int WM = 2, WN = T == 256 ? 4 : 2;
    muon_product_kernel<MODE, T, T, WM, WN><<<dim3((unsigned)blocks), dim3(WM * WN * 64), 0, s>>>(b, st, out, ov);
}

template <int T>
void launch_steps(MuonBuffers &b, MuonStep st, int steps, int count, uint16_t *out, const MuonView &ov, hipStream_t s)
{
    for (int k = 0; k < steps; ++k) {
        launch_product<kModeA, T>(b, st, count, out, ov, s);
        launch_product<kModeB, T>(b, st, count, out, ov, s);
        if (k + 1 < steps)
            launch_product<kModeX, T>(b, st, count, out, ov, s);
        else
            launch_product<kModeOut, T>(b, st, count, out, ov, s);
        st.cur ^= 1;
    }
}

template <typename T>
void launch_load(const void *g, const MuonView &gv, const MuonBuffers &b, int count, float eps, hipStream_t s)
{
    const T *p = reinterpret_cast<const T *>(g);
    muon_norm_kernel<T><<<dim3(kNormParts, (unsigned)count), dim3(256), 0, s>>>(p, gv, b.part);
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
    if (count * (p.mp / p.tile) * (p.np / p.tile) > INT32_MAX)
        return MXQ_ERR_INVALID_ARG;

    MuonBuffers buf;
    buf.mp = (int)p.mp;
    buf.np = (int)p.np;
    buf.part = reinterpret_cast<double *>(workspace);
    const int64_t nx = count * p.mp * p.np, na = count * p.mp * p.mp;
    buf.xh = reinterpret_cast<_Float16 *>(buf.part + count * kNormParts);
    buf.xl = buf.xh + nx;
    buf.xt[0] = buf.xl + nx;
    buf.xt[1] = buf.xt[0] + nx;
    buf.oh = buf.xt[1] + nx;
    buf.ol = buf.oh + na;
    buf.bo = buf.ol + na;
    buf.d = reinterpret_cast<float *>(buf.bo + na);
    buf.db = buf.d + count * p.mp;

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
        muon_copy_kernel<<<dim3((unsigned)((gv.n + 255) / 256), (unsigned)gv.m, (unsigned)count), dim3(256), 0, s>>>(
            buf, st.out_scale, out, ov);
    else if (p.tile == 256)
        launch_steps<256>(buf, st, steps, (int)count, out, ov, s);
    else if (p.tile == 128)
        launch_steps<128>(buf, st, steps, (int)count, out, ov, s);
    else
        launch_steps<64>(buf, st, steps, (int)count, out, ov, s);
    return launch_status();
}

}  // extern "C"
