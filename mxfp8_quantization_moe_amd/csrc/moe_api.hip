// C entry points of the mixture-of-experts routing operators: argument
// checks, the choice of a kernel variant and the launches.  No allocation, no
// synchronisation, no read-back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mxq.h"
#include "api_common.hpp"
#include "moe_route_kernels.hpp"
#include "moe_rows_kernels.hpp"

namespace {

using namespace mxq;

bool dtype_ok(int32_t dtype) { return dtype == MXQ_BF16 || dtype == MXQ_F32; }
uintptr_t dtype_size(int32_t dtype) { return dtype == MXQ_BF16 ? 2 : 4; }

// rows of the grouped buffer, whatever the router picks: every slot, and the
// padding of each expert that can have a slot
int64_t row_capacity(int64_t tokens, int64_t k, int64_t experts, int64_t align)
{
    const int64_t slots = tokens * k;
    return slots + std::min(experts, slots) * (align - 1);
}

constexpr int64_t kMaxWidth = 1 << 30;  // element numbers of a row and a piece more fit 32 bits

bool plan_ok(int64_t tokens, int32_t k, int32_t experts)
{
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= MXQ_MAX_GROUPS && k >= 1 &&
           k <= MXQ_MAX_TOP_K && k <= experts && tokens * k <= INT32_MAX;
}

// tokens of a run: whole rounds of kRouteTile tokens, at most kRouteMaxBlocks
// runs, one for each CU (65536 x 256 bf16 logits 41 us, 60 with 128 runs)
int64_t route_run(int64_t tokens)
{
    const int64_t rounds = (tokens + kRouteTile - 1) / kRouteTile;
    return (rounds + kRouteMaxBlocks - 1) / kRouteMaxBlocks * kRouteTile;
}

int64_t route_runs(int64_t tokens)
{
    return tokens > 0 ? (tokens + route_run(tokens) - 1) / route_run(tokens) : 0;
}

// a single run needs no workspace
int64_t route_bytes(int64_t tokens, int64_t experts)
{
    const int64_t runs = route_runs(tokens);
    return runs <= 1 ? 0 : experts * 8 + runs * (2 * experts + 2) * 4;
}

// Lanes per token, experts per lane and threads by the number of experts.
// Sixteen lanes reduce within a DPP row, without LDS permutes; more experts
// per lane share those steps among more tokens of a wave.  With a whole wave
// per token instead: 262144 x 8 bf16 logits 28 -> 103 us (gradient 12 -> 99),
// x 64 70 -> 148 (31 -> 98), 65536 x 256 41 -> 68 (21 -> 32).
template <typename F>
void by_experts(int experts, F &&f)
{
    auto go = [&](auto l, auto v, auto t) { f(l, v, t); };
#define MXQ_CONFIG(L, V, THREADS)                                                                              \
    go(std::integral_constant<int, L>(), std::integral_constant<int, V>(), std::integral_constant<int, THREADS>())
    if (experts <= 8)
        MXQ_CONFIG(8, 1, 512);
    else if (experts <= 32)
        MXQ_CONFIG(8, 4, 512);
    else if (experts <= 64)
        MXQ_CONFIG(16, 4, 1024);
    else if (experts <= 128)
        MXQ_CONFIG(16, 8, 1024);
    else if (experts <= 256)
        MXQ_CONFIG(16, 16, 1024);
    else if (experts <= 512)
        MXQ_CONFIG(32, 16, 1024);
    else if (experts <= 1024)
        MXQ_CONFIG(64, 16, 1024);
    else
        MXQ_CONFIG(64, 64, 256);
#undef MXQ_CONFIG
}

// runs * experts up to which one kernel does the scan and the placement: a
// launch less against every workgroup reading all counts.  On the GPU, whole
// call: 2048 counts (16384 tokens, 8 experts) 10.3 against 13.4 us, 3965 16.3
// against 17.5, 4096 21.7 against 21.8, 8192 17.6 against 16.2, 16384 28.3
// against 19.0.
constexpr int64_t kFinishCounts = 4096;

template <typename T>
mxq_status run_route(const void *logits, int64_t sl, int tokens, int experts, const uint8_t *mask, int k,
                     int renorm, int align, int32_t *ids, float *weights, int32_t *rows, float *lse,
                     const RouteResults &out, void *workspace, hipStream_t st)
{
    const int run = (int)std::max<int64_t>(route_run(tokens), kRouteTile), nruns = (int)route_runs(tokens);
    RouteWorkspace ws = {};
    if (nruns > 1) {
        ws.balance = reinterpret_cast<double *>(workspace);
        ws.counts = reinterpret_cast<int32_t *>(ws.balance + experts);
        ws.probs = reinterpret_cast<float *>(ws.counts + (int64_t)nruns * experts);
        ws.z = ws.probs + (int64_t)nruns * experts;
        ws.live = reinterpret_cast<int32_t *>(ws.z + nruns);
    }
    const size_t lds = (size_t)experts * 12 + (size_t)kRouteTile * 6 * k;
    by_experts(experts, [&](auto l, auto v, auto t) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value, THREADS = decltype(t)::value;
        auto go = [&](auto kernel) {
            kernel<<<dim3((unsigned)std::max(nruns, 1)), dim3(THREADS), lds, st>>>(
                reinterpret_cast<const T *>(logits), sl, tokens, experts, mask, k, renorm, align, run, ids, weights,
                rows, lse, ws, out);
        };
        if (k <= 8)
            nruns <= 1 ? go(moe_route_kernel<T, L, V, true, THREADS, true>)
                       : go(moe_route_kernel<T, L, V, true, THREADS, false>);
        else
            nruns <= 1 ? go(moe_route_kernel<T, L, V, false, THREADS, true>)
                       : go(moe_route_kernel<T, L, V, false, THREADS, false>);
    });
    if (nruns > 1 && (int64_t)nruns * experts <= kFinishCounts) {
        const int parts = std::max(1, kPlaceThreads / experts);
        moe_finish_kernel<<<dim3((unsigned)(nruns + 1)), dim3(kPlaceThreads),
                            (size_t)parts * experts * 8 + (size_t)experts * 8, st>>>(
            tokens, experts, k, align, run, nruns, ids, rows, ws, out);
    } else if (nruns > 1) {
        moe_scan_kernel<<<dim3((unsigned)((experts + kScanExperts - 1) / kScanExperts)), dim3(kScanThreads), 0, st>>>(
            experts, nruns, ws, out);
        moe_place_kernel<<<dim3((unsigned)(nruns + 1)), dim3(kPlaceThreads), (size_t)experts * 4, st>>>(
            tokens, experts, k, align, run, nruns, ids, rows, ws, out);
    }
    return launch_status();
}

template <typename T>
mxq_status run_route_backward(const void *logits, int64_t sl, int tokens, int experts, int k, int renorm,
                              const int32_t *ids, const float *weights, const float *lse, const int32_t *counts,
                              const int32_t *live, const float *gw, const float *gl, void *dl, int64_t sd,
                              hipStream_t st)
{
    by_experts(experts, [&](auto l, auto v, auto) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        const int per = 256 / L;
        const int64_t blocks = std::min<int64_t>(((int64_t)tokens + per - 1) / per, 1 << 20);
        moe_route_backward_kernel<T, L, V><<<dim3((unsigned)blocks), dim3(256), (size_t)256 * route_row_step(V) * 4, st>>>(
            reinterpret_cast<const T *>(logits), sl, tokens, experts, k, renorm, ids, weights, lse, counts, live,
            gw, gl, reinterpret_cast<T *>(dl), sd);
    });
    return launch_status();
}

// workgroups that clear the rows without a slot: enough to keep the memory
// busy when masked tokens leave a long tail (16384 tokens of 4096 bf16 over 2
// slots, half of them masked: dispatch 59.2 us, 69.1 with 128)
int clear_blocks(int64_t capacity) { return (int)std::min<int64_t>(capacity, 1024); }

// pieces per lane of a dispatch: up to four, fewer for rows that short.  The
// slots' rows are read from memory once for four times the stores: 8192 tokens
// of 4096 bf16 over 8 slots 119 us with four, 127 with one; 32768 of 512 46.7
// us with one, 53.6 with four.
template <typename T>
int pieces_per_lane(int64_t width)
{
    int u = 4;
    while (u > 1 && width <= 64 * Piece<T>::N * (u / 2))
        u /= 2;
    return u;
}

// from here on a call's loads carry the nontemporal hint (see ld_piece): between
// the 100 MB that lose by it and the 200 MB that are even or gain
constexpr int64_t kStreamBytes = 160 << 20;
template <typename T>
bool streams(int64_t tokens, int64_t width, int k)
{
    return tokens * width * (k + 1) * (int64_t)sizeof(T) >= kStreamBytes;
}

// Workgroups of one launch: a grid ends before 2^32 threads.  More tokens than
// that takes are passed in several launches, `launch(t0, n)` for n of them
// from t0 on, the first also without tokens.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 32) / kRowsThreads - 1;
template <typename F>
mxq_status in_launches(int64_t tokens, int64_t per, F &&launch)
{
    int64_t t0 = 0;
    do {
        launch(t0, (int)std::min(per, tokens - t0));
        t0 += per;
    } while (t0 < tokens);
    return launch_status();
}

template <typename T, int U>
mxq_status run_dispatch(const void *x, int64_t sx, int tokens, int width, const int32_t *rows, int k,
                        const int32_t *counts, const int32_t *offs, int experts, void *out, int64_t ld,
                        int capacity, hipStream_t st)
{
    const int64_t span = 64 * Piece<T>::N * U, chunks = (width + span - 1) / span;
    auto kernel = streams<T>(tokens, width, k) ? moe_dispatch_kernel<T, U, true> : moe_dispatch_kernel<T, U, false>;
    return in_launches(tokens, (kMaxBlocks - clear_blocks(capacity)) * 4 / chunks, [&](int64_t t0, int n) {
        const int64_t work = (n * chunks + 3) / 4, clear = t0 ? 0 : clear_blocks(capacity);
        kernel<<<dim3((unsigned)(work + clear)), dim3(kRowsThreads), 0, st>>>(
            reinterpret_cast<const T *>(x) + t0 * sx, sx, n, width, rows + t0 * k, k, counts, offs, experts,
            reinterpret_cast<T *>(out), ld, capacity, (int)chunks, (int)work);
    });
}

template <typename T, int KB>
mxq_status run_combine(const void *in, int64_t ld, int capacity, int width, const int32_t *rows,
                       const float *weights, int k, const void *resid, int64_t sr, void *y, int64_t sy, int tokens,
                       hipStream_t st)
{
    const int64_t span = 64 * Piece<T>::N, chunks = (width + span - 1) / span;
    auto kernel = streams<T>(tokens, width, k) ? moe_combine_kernel<T, KB, true> : moe_combine_kernel<T, KB, false>;
    return in_launches(tokens, kMaxBlocks * 4 / chunks, [&](int64_t t0, int n) {
        const int64_t work = (n * chunks + 3) / 4;
        kernel<<<dim3((unsigned)work), dim3(kRowsThreads), 0, st>>>(
            reinterpret_cast<const T *>(in), ld, capacity, width, rows + t0 * k, weights ? weights + t0 * k : nullptr,
            k, resid ? reinterpret_cast<const T *>(resid) + t0 * sr : nullptr, sr, reinterpret_cast<T *>(y) + t0 * sy,
            sy, n, (int)chunks);
    });
}

template <typename T, int NW, int KB>
mxq_status run_combine_backward(const void *dy, int64_t sy, int tokens, int width, const void *in, int64_t ld,
                                const int32_t *rows, const float *weights, int k, const int32_t *counts,
                                const int32_t *offs, int experts, int capacity, void *out, int64_t ldo, float *dw,
                                hipStream_t st)
{
    constexpr int TPB = kRowsThreads / 64 / NW;
    // rows read and written
    auto kernel = streams<T>(tokens, width, 2 * k) ? moe_combine_backward_kernel<T, NW, KB, true>
                                                   : moe_combine_backward_kernel<T, NW, KB, false>;
    return in_launches(tokens, (kMaxBlocks - clear_blocks(capacity)) * TPB, [&](int64_t t0, int n) {
        const int64_t work = (n + TPB - 1) / TPB, clear = t0 ? 0 : clear_blocks(capacity);
        kernel<<<dim3((unsigned)(work + clear)), dim3(kRowsThreads), 0, st>>>(
            reinterpret_cast<const T *>(dy) + t0 * sy, sy, n, width, reinterpret_cast<const T *>(in), ld, rows + t0 * k,
            weights + t0 * k, k, counts, offs, experts, capacity, reinterpret_cast<T *>(out), ldo, dw + t0 * k,
            (int)work);
    });
}

// a 2-D operand of rows of `width` unit-stride elements, `n` of them
bool rows_ok(const void *p, int32_t dtype, int64_t n, int64_t stride, bool writes, int64_t width)
{
    if (n > 0 && width > 0 && !p)
        return false;
    return aligned_to(p, dtype_size(dtype)) && stride >= 0 && (!writes || n <= 1 || stride >= width);
}

}  // namespace

extern "C" {

int64_t mxq_moe_row_capacity(int64_t tokens, int32_t top_k, int32_t num_experts, int32_t align)
{
    if (!plan_ok(tokens, top_k, num_experts) || align < 1 || align > MXQ_MAX_GROUP_ALIGN)
        return -1;
    const int64_t c = row_capacity(tokens, top_k, num_experts, align);
    return c <= INT32_MAX ? c : -1;
}

int64_t mxq_moe_route_workspace_bytes(int64_t tokens, int32_t num_experts, int32_t top_k)
{
    if (!plan_ok(tokens, top_k, num_experts))
        return -1;
    return route_bytes(tokens, num_experts);
}

mxq_status mxq_moe_route(const void *logits, int32_t dtype, int64_t tokens, int32_t num_experts, int64_t sl_t,
                         int64_t sl_e, const uint8_t *token_mask, int32_t top_k, int32_t renormalize, int32_t align,
                         int32_t *ids, float *weights, int32_t *rows, float *lse, int32_t *counts, int32_t *offs,
                         float *mean_prob, float *losses, int32_t *live, void *workspace, int64_t workspace_bytes,
                         void *stream)
{
    if (!dtype_ok(dtype) || mxq_moe_row_capacity(tokens, top_k, num_experts, align) < 0 ||
        (renormalize != 0 && renormalize != 1))
        return MXQ_ERR_INVALID_ARG;
    if (!counts || !offs || !mean_prob || !losses || !live)
        return MXQ_ERR_INVALID_ARG;
    if (tokens > 0 && (!logits || !ids || !weights || !rows || !lse))
        return MXQ_ERR_INVALID_ARG;
    if (num_experts > 1 && sl_e != 1)
        return MXQ_ERR_UNSUPPORTED;
    if (sl_t < 0 || !aligned_to(logits, dtype_size(dtype)) || !aligned_to(workspace, 8))
        return MXQ_ERR_INVALID_ARG;
    const int64_t need = route_bytes(tokens, num_experts);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return MXQ_ERR_WORKSPACE;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return (dtype == MXQ_BF16 ? run_route<uint16_t> : run_route<float>)(
        logits, sl_t, (int)tokens, num_experts, token_mask, top_k, renormalize, align, ids, weights, rows, lse,
        RouteResults{counts, offs, mean_prob, losses, live}, workspace, st);
}

mxq_status mxq_moe_route_backward(const void *logits, int32_t dtype, int64_t tokens, int32_t num_experts,
                                  int64_t sl_t, int64_t sl_e, int32_t top_k, int32_t renormalize,
                                  const int32_t *ids, const float *weights, const float *lse, const int32_t *counts,
                                  const int32_t *live, const float *grad_weights, const float *grad_losses,
                                  void *grad_logits, int64_t sg_t, int64_t sg_e, void *stream)
{
    if (!dtype_ok(dtype) || !plan_ok(tokens, top_k, num_experts) || (renormalize != 0 && renormalize != 1))
        return MXQ_ERR_INVALID_ARG;
    if (tokens == 0)
        return MXQ_OK;
    if (!logits || !lse || !grad_logits || (grad_weights && (!ids || !weights)) ||
        (grad_losses && (!counts || !live)))
        return MXQ_ERR_INVALID_ARG;
    if (num_experts > 1 && (sl_e != 1 || sg_e != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (sl_t < 0 || !aligned_to(logits, dtype_size(dtype)) ||
        !rows_ok(grad_logits, dtype, tokens, sg_t, true, num_experts))
        return MXQ_ERR_INVALID_ARG;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return (dtype == MXQ_BF16 ? run_route_backward<uint16_t> : run_route_backward<float>)(
        logits, sl_t, (int)tokens, num_experts, top_k, renormalize, ids, weights, lse, counts, live, grad_weights,
        grad_losses, grad_logits, sg_t, st);
}

mxq_status mxq_moe_dispatch(const void *x, int32_t dtype, int64_t tokens, int64_t width, int64_t sx_t, int64_t sx_c,
                            const int32_t *rows, int32_t top_k, const int32_t *counts, const int32_t *offs,
                            int32_t num_experts, void *xg, int64_t capacity, int64_t sg_r, int64_t sg_c,
                            void *stream)
{
    if (!dtype_ok(dtype) || !plan_ok(tokens, top_k, num_experts) || width < 0 || width > kMaxWidth || capacity < 0 ||
        capacity > INT32_MAX || !counts || !offs || (tokens > 0 && !rows))
        return MXQ_ERR_INVALID_ARG;
    if (width > 1 && (sx_c != 1 || sg_c != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (!rows_ok(x, dtype, tokens, sx_t, false, width) || !rows_ok(xg, dtype, capacity, sg_r, true, width))
        return MXQ_ERR_INVALID_ARG;
    if (width == 0 || capacity == 0)
        return MXQ_OK;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
#define MXQ_DISPATCH(T, U)                                                                                        \
    run_dispatch<T, U>(x, sx_t, (int)tokens, (int)width, rows, top_k, counts, offs, num_experts, xg, sg_r,        \
                       (int)capacity, st)
#define MXQ_DISPATCH_T(T)                                                                                         \
    do {                                                                                                          \
        const int u = pieces_per_lane<T>(width);                                                                  \
        return u == 4 ? MXQ_DISPATCH(T, 4) : u == 2 ? MXQ_DISPATCH(T, 2) : MXQ_DISPATCH(T, 1);                    \
    } while (0)
    if (dtype == MXQ_BF16)
        MXQ_DISPATCH_T(uint16_t);
    MXQ_DISPATCH_T(float);
#undef MXQ_DISPATCH_T
#undef MXQ_DISPATCH
}

mxq_status mxq_moe_combine(const void *yg, int32_t dtype, int64_t capacity, int64_t width, int64_t sg_r, int64_t sg_c,
                           const int32_t *rows, const float *weights, int32_t top_k, const void *residual,
                           int64_t sr_t, int64_t sr_c, void *y, int64_t sy_t, int64_t sy_c, int64_t tokens,
                           void *stream)
{
    if (!dtype_ok(dtype) || !plan_ok(tokens, top_k, MXQ_MAX_GROUPS) || width < 0 || width > kMaxWidth ||
        capacity < 0 || capacity > INT32_MAX || (tokens > 0 && !rows))
        return MXQ_ERR_INVALID_ARG;
    if (width > 1 && (sg_c != 1 || sy_c != 1 || (residual && sr_c != 1)))
        return MXQ_ERR_UNSUPPORTED;
    if (!rows_ok(yg, dtype, capacity, sg_r, false, width) || !rows_ok(y, dtype, tokens, sy_t, true, width) ||
        (residual && !rows_ok(residual, dtype, tokens, sr_t, false, width)))
        return MXQ_ERR_INVALID_ARG;
    if (width == 0 || tokens == 0)
        return MXQ_OK;
    const int k = capacity > 0 ? top_k : 0;  // an empty buffer: every slot is empty
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
#define MXQ_COMBINE(T, KB)                                                                                        \
    run_combine<T, KB>(yg, sg_r, (int)capacity, (int)width, rows, weights, k, residual, sr_t, y, sy_t,            \
                       (int)tokens, st)
    // all of a token's slots at once, up to eight
#define MXQ_COMBINE_T(T) return k <= 2 ? MXQ_COMBINE(T, 2) : k <= 4 ? MXQ_COMBINE(T, 4) : MXQ_COMBINE(T, 8)
    if (dtype == MXQ_BF16)
        MXQ_COMBINE_T(uint16_t);
    MXQ_COMBINE_T(float);
#undef MXQ_COMBINE_T
#undef MXQ_COMBINE
}

mxq_status mxq_moe_combine_backward(const void *grad_y, int32_t dtype, int64_t tokens, int64_t width, int64_t sy_t,
                                    int64_t sy_c, const void *yg, int64_t sg_r, int64_t sg_c, const int32_t *rows,
                                    const float *weights, int32_t top_k, const int32_t *counts, const int32_t *offs,
                                    int32_t num_experts, int64_t capacity, void *grad_yg, int64_t sd_r, int64_t sd_c,
                                    float *grad_weights, void *stream)
{
    if (!dtype_ok(dtype) || !plan_ok(tokens, top_k, num_experts) || width < 0 || width > kMaxWidth || capacity < 0 ||
        capacity > INT32_MAX || !counts || !offs || (tokens > 0 && (!rows || !weights || !grad_weights)))
        return MXQ_ERR_INVALID_ARG;
    if (width > 1 && (sy_c != 1 || sg_c != 1 || sd_c != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (!rows_ok(grad_y, dtype, tokens, sy_t, false, width) || !rows_ok(yg, dtype, capacity, sg_r, false, width) ||
        !rows_ok(grad_yg, dtype, capacity, sd_r, true, width))
        return MXQ_ERR_INVALID_ARG;
    if (tokens == 0 && (capacity == 0 || width == 0))
        return MXQ_OK;
    // an empty buffer: every slot is empty and its loads (unused) go to the
    // gradient's first row instead
    const void *in = capacity > 0 ? yg : grad_y;
    const int64_t ld = capacity > 0 ? sg_r : 0;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
#define MXQ_COMBINE_BWD(T, NW, KB)                                                                                \
    run_combine_backward<T, NW, KB>(grad_y, sy_t, (int)tokens, (int)width, in, ld, rows, weights, top_k, counts,  \
                                    offs, num_experts, (int)capacity, grad_yg, sd_r, grad_weights, st)
    // a wave per token for rows of up to two loads per lane, else a workgroup:
    // over 2 slots 65536 tokens of 1024 bf16 106 us (130 with a workgroup per
    // token), 16384 of 2048 55 us (63 with a wave)
#define MXQ_COMBINE_BWD_T(T)                                                                                      \
    do {                                                                                                          \
        const bool narrow = width <= 64 * 2 * Piece<T>::N;                                                        \
        if (top_k <= 2)                                                                                           \
            return narrow ? MXQ_COMBINE_BWD(T, 1, 2) : MXQ_COMBINE_BWD(T, 4, 2);                                  \
        if (top_k <= 4)                                                                                           \
            return narrow ? MXQ_COMBINE_BWD(T, 1, 4) : MXQ_COMBINE_BWD(T, 4, 4);                                  \
        return narrow ? MXQ_COMBINE_BWD(T, 1, 8) : MXQ_COMBINE_BWD(T, 4, 8);                                      \
    } while (0)
    if (dtype == MXQ_BF16)
        MXQ_COMBINE_BWD_T(uint16_t);
    MXQ_COMBINE_BWD_T(float);
#undef MXQ_COMBINE_BWD_T
#undef MXQ_COMBINE_BWD
}

}  // extern "C"
