// C entry points of the mixture-of-experts layer for a few tokens: argument
// checks, the workspace's layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mxq.h"
#include "api_common.hpp"
#include "moe_layer_kernels.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxDim = 65536;

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

bool sizes_ok(int64_t tokens, int64_t width, int64_t hidden, int32_t experts, int32_t k)
{
    return tokens >= 0 && tokens <= MXQ_LAYER_MAX_TOKENS && width >= 0 && width <= kMaxDim && hidden >= 0 &&
           hidden <= kMaxDim && experts >= 1 && experts <= MXQ_LAYER_MAX_EXPERTS && k >= 1 && k <= MXQ_MAX_TOP_K &&
           k <= experts;
}

// Workgroups per 8 rows of the down product, each with a part of its sums: up to
// 256 in all, with some steps for every wave.  From 129 blocks on, widths above
// 1024, there is one part; the limits were not measured on both sides.
int layer_splits(int64_t tokens, int64_t width, int64_t hidden, int32_t experts, int32_t k)
{
    const int64_t blocks = (width + 7) / 8, steps = std::min<int64_t>(experts, tokens * k) * ((hidden + 63) / 64);
    int s = 1;
    while (s < 8 && blocks * s <= 128 && steps >= 8 * kDownWaves * s)
        s *= 2;
    return s;
}

struct LayerLayout {
    int64_t ids, share, active, begin, order, hi, lo, parts, bytes;
    int hp, splits, most;
};

LayerLayout layer_layout(int64_t tokens, int64_t width, int64_t hidden, int32_t experts, int32_t k)
{
    LayerLayout l;
    const int64_t slots = tokens * k;
    l.hp = (int)round_up(hidden, 8);
    l.splits = layer_splits(tokens, width, hidden, experts, k);
    l.most = (int)std::min<int64_t>(experts, slots);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += round_up(bytes, 16);
        return from;
    };
    l.ids = take(slots * 4);
    l.share = take(slots * 4);
    l.active = take(l.most * 4);
    l.begin = take((l.most + 2) * 4);
    l.order = take(slots * 4);
    l.hi = take(slots * l.hp * 2);
    l.lo = take(slots * l.hp * 2);
    l.parts = take(l.splits > 1 ? l.splits * tokens * width * 4 : 0);
    l.bytes = at;
    return l;
}

// weights of a format, unit stride along the summed dim
mxq_status weights_status(const void *w, const uint8_t *scales, int32_t format, int64_t se, int64_t sr, int64_t sc,
                          int64_t sse, int64_t ssr, int64_t ssb, int64_t cols, const void *bias, int32_t bias_dtype,
                          int64_t sb)
{
    if (!w || (bias && ((bias_dtype != MXQ_BF16 && bias_dtype != MXQ_F32) ||
                        !aligned_to(bias, bias_dtype == MXQ_BF16 ? 2 : 4) || sb < 0)))
        return MXQ_ERR_INVALID_ARG;
    if (format == MXQ_WEIGHTS_MX && (!scales || cols % 32))
        return MXQ_ERR_INVALID_ARG;
    if (cols > 1 && (sc != 1 || (format == MXQ_WEIGHTS_MX && cols > 32 && ssb != 1)))
        return MXQ_ERR_UNSUPPORTED;
    if (se < 0 || sr < 0)
        return MXQ_ERR_INVALID_ARG;
    if (format == MXQ_WEIGHTS_MX ? !aligned16(w) || se % 16 || sr % 16 || sse < 0 || ssr < 0 : !aligned_to(w, 2))
        return MXQ_ERR_INVALID_ARG;
    return MXQ_OK;
}

// 16 rows of U per workgroup where 32 would leave fewer than four workgroups per
// CU, else 32, for half the searches and half the loads of the tokens' values: 8
// tokens in MXFP8 over 256 experts of 2048 x 768 84 us a call (88 with 16).
template <typename T, bool MX, bool GATED>
void launch_up(const LayerArgs &a, hipStream_t st)
{
    auto grid = [&](int fragments) {
        const int rows = (GATED ? 8 : 16) * fragments;
        return dim3((unsigned)((a.hidden + rows - 1) / rows), (unsigned)a.most);
    };
    auto go = [&](auto kernel, int fragments) { kernel<<<grid(fragments), dim3(kLayerThreads), 0, st>>>(a); };
    if (a.tokens == 1)
        go(layer_up_one_kernel<T, MX, GATED>, 1);
    else if (a.tokens <= 16)
        (int64_t)grid(2).x * a.most < 1024 ? go(layer_up_kernel<MX, GATED, 1, 1>, 1) : go(layer_up_kernel<MX, GATED, 2, 1>, 2);
    else
        a.tokens <= 32 ? go(layer_up_kernel<MX, GATED, 2, 2>, 2) : go(layer_up_kernel<MX, GATED, 2, 4>, 2);
}

template <bool MX>
void launch_down(const LayerArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.width + 7) / 8), (unsigned)a.splits);
    constexpr int WAVES = MX ? kDownWavesMx : kDownWaves;
    const size_t lds = ((size_t)WAVES * 2 * a.tokens * 8 + 2 * a.most + 1 + a.tokens * a.k) * 4;
    auto go = [&](auto kernel) { kernel<<<grid, dim3(WAVES * 64), lds, st>>>(a); };
    a.hidden % (2 * WeightStep<MX>::K) == 0 ? go(layer_down_kernel<MX, true>) : go(layer_down_kernel<MX, false>);
}

template <typename T, bool MX>
void launch_layer(const LayerArgs &a, int gated, hipStream_t st)
{
    if (a.tokens > 1)
        layer_select_kernel<T><<<dim3(1), dim3(kSelectThreads), 0, st>>>(a);
    gated ? launch_up<T, MX, true>(a, st) : launch_up<T, MX, false>(a, st);
    launch_down<MX>(a, st);
    if (a.splits > 1)
        layer_join_kernel<<<dim3((unsigned)((a.width + kLayerThreads - 1) / kLayerThreads), (unsigned)a.tokens),
                            dim3(kLayerThreads), 0, st>>>(a);
}

}  // namespace

extern "C" {

int64_t mxq_moe_layer_workspace_bytes(int64_t tokens, int64_t width, int64_t hidden, int32_t num_experts, int32_t top_k)
{
    return sizes_ok(tokens, width, hidden, num_experts, top_k) ? layer_layout(tokens, width, hidden, num_experts, top_k).bytes : -1;
}

mxq_status mxq_moe_layer(const uint16_t *x, int64_t tokens, int64_t width, int64_t sx_t, int64_t sx_c, const void *logits,
                         int32_t logits_dtype, int32_t num_experts, int64_t sl_t, int64_t sl_e, const uint8_t *token_mask,
                         int32_t top_k, int32_t renormalize, int64_t hidden, int32_t format, const void *up,
                         const uint8_t *up_scales, int64_t su_e, int64_t su_r, int64_t su_c, int64_t sus_e, int64_t sus_r,
                         int64_t sus_b, const void *bias_up, const void *down, const uint8_t *down_scales, int64_t sd_e,
                         int64_t sd_r, int64_t sd_c, int64_t sds_e, int64_t sds_r, int64_t sds_b, const void *bias_down,
                         int32_t bias_dtype, int64_t sbu_e, int64_t sbd_e, int32_t activation, int32_t gated,
                         const uint16_t *residual, int64_t sr_t, int64_t sr_c, uint16_t *y, int64_t sy_t, int64_t sy_c,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(tokens, width, hidden, num_experts, top_k) || (logits_dtype != MXQ_BF16 && logits_dtype != MXQ_F32) ||
        (renormalize != 0 && renormalize != 1) || (format != MXQ_WEIGHTS_BF16 && format != MXQ_WEIGHTS_MX) ||
        activation < MXQ_ACT_NONE || activation > MXQ_ACT_SILU || (gated != 0 && gated != 1) || !aligned16(workspace))
        return MXQ_ERR_INVALID_ARG;
    if (tokens == 0 || width == 0)
        return MXQ_OK;
    if (!x || !logits || !y || !aligned_to(x, 2) || !aligned_to(y, 2) || !aligned_to(residual, 2) ||
        !aligned_to(logits, logits_dtype == MXQ_BF16 ? 2 : 4) || sx_t < 0 || sl_t < 0 || sr_t < 0 ||
        (tokens > 1 && sy_t < width))
        return MXQ_ERR_INVALID_ARG;
    if ((width > 1 && (sx_c != 1 || sy_c != 1 || (residual && sr_c != 1))) || (num_experts > 1 && sl_e != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (hidden > 0) {
        mxq_status s = weights_status(up, up_scales, format, su_e, su_r, su_c, sus_e, sus_r, sus_b, width, bias_up, bias_dtype, sbu_e);
        if (s == MXQ_OK)
            s = weights_status(down, down_scales, format, sd_e, sd_r, sd_c, sds_e, sds_r, sds_b, hidden, bias_down, bias_dtype, sbd_e);
        if (s != MXQ_OK)
            return s;
    } else if (bias_down && ((bias_dtype != MXQ_BF16 && bias_dtype != MXQ_F32) ||
                             !aligned_to(bias_down, bias_dtype == MXQ_BF16 ? 2 : 4) || sbd_e < 0)) {
        return MXQ_ERR_INVALID_ARG;
    }
    const LayerLayout l = layer_layout(tokens, width, hidden, num_experts, top_k);
    if (!workspace || workspace_bytes < l.bytes)
        return MXQ_ERR_WORKSPACE;
    char *ws = reinterpret_cast<char *>(workspace);
    LayerArgs a = {};
    a.x = x;
    a.sx = sx_t;
    a.logits = logits;
    a.sl = sl_t;
    a.mask = token_mask;
    a.tokens = (int)tokens;
    a.width = (int)width;
    a.hidden = (int)hidden;
    a.experts = num_experts;
    a.k = top_k;
    a.renorm = renormalize;
    a.act = activation;
    a.up = {up, su_e, su_r, up_scales, sus_e, sus_r, bias_up, sbu_e, bias_dtype == MXQ_F32};
    a.down = {down, sd_e, sd_r, down_scales, sds_e, sds_r, bias_down, sbd_e, bias_dtype == MXQ_F32};
    a.resid = residual;
    a.sr = sr_t;
    a.y = y;
    a.sy = sy_t;
    a.ids = reinterpret_cast<int32_t *>(ws + l.ids);
    a.share = reinterpret_cast<float *>(ws + l.share);
    a.active = reinterpret_cast<int32_t *>(ws + l.active);
    a.begin = reinterpret_cast<int32_t *>(ws + l.begin);
    a.order = reinterpret_cast<int32_t *>(ws + l.order);
    a.most = l.most;
    a.hi = reinterpret_cast<uint16_t *>(ws + l.hi);
    a.lo = reinterpret_cast<uint16_t *>(ws + l.lo);
    a.hp = l.hp;
    a.parts = reinterpret_cast<float *>(ws + l.parts);
    a.splits = l.splits;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool mx = format == MXQ_WEIGHTS_MX;
    if (hidden == 0) {
        // nothing to multiply: biases and residual alone
        a.splits = 0;
        logits_dtype == MXQ_BF16 ? layer_select_kernel<uint16_t><<<dim3(1), dim3(kSelectThreads), 0, st>>>(a)
                                 : layer_select_kernel<float><<<dim3(1), dim3(kSelectThreads), 0, st>>>(a);
        layer_join_kernel<<<dim3((unsigned)((width + kLayerThreads - 1) / kLayerThreads), (unsigned)tokens),
                            dim3(kLayerThreads), 0, st>>>(a);
    } else if (logits_dtype == MXQ_BF16) {
        mx ? launch_layer<uint16_t, true>(a, gated, st) : launch_layer<uint16_t, false>(a, gated, st);
    } else {
        mx ? launch_layer<float, true>(a, gated, st) : launch_layer<float, false>(a, gated, st);
    }
    return launch_status();
}

}  // extern "C"
