// The router of a mixture of experts: softmax, the k largest logits, the
// per-expert counts and group ends, the row of every (token, slot) in the
// grouped layout, the balance and z losses, and the logits' gradient.
//
// With l the logits of a live token (token mask set, some logit > -inf) and
// n the number of live tokens:
//   lse_t = log sum_e exp l_te        p_te = exp(l_te - lse_t)
//   ids_t = indices of the k largest logits, descending, ties to the lower
//           index; -inf (and NaN) is never taken and leaves an empty slot
//   w_tj  = p_{t, ids_tj}, or that over the sum of the token's slots
//   c_e   = number of slots that name e
//   offs_e = sum_{e' <= e} ceil(c_e' / align) * align
//   rows_tj = offs_{e-1} + number of earlier tokens that have e in a slot
//   P_e = 1/n sum_t p_te     balance = E sum_e c_e/(n k) P_e
//   z = 1/n sum_t lse_t^2
//
// Two kernels.  The first gives each workgroup a run of tokens (at most
// kRouteMaxBlocks runs): L lanes hold a token's logits, V consecutive ones
// per lane, so the whole row stays in registers and every reduction is a few
// cross-lane steps.  64 tokens at a time set their bits in one 64-bit mask
// per expert in LDS; a slot's rank among the run's slots of its expert is
// then a population count, whatever order the lanes ran in, and no atomic
// result depends on an order.  The second kernel turns the runs' counts into
// ranks over all tokens and into the per-expert results.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_rows_kernels.hpp"
#include "mxq_device.hpp"
#include "wave_ops.hpp"

namespace mxq {

constexpr int kRouteTile = 64;        // tokens that share one round of bit masks
constexpr int kRouteMaxBlocks = 256;  // runs of tokens (workgroups of the first kernel)
constexpr int kNoExpert = 0xffff;
constexpr int kRankThreads = 1024;    // workgroups of the second kernel

// fp32 -> uint32 whose unsigned order is the float order (-0 equals +0: adding
// zero makes it +0); NaN and -inf -> 0
__device__ __forceinline__ uint32_t route_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v > -INFINITY ? b ^ (b >> 31 ? 0xffffffffu : 0x80000000u) : 0u;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int m = 1; m < L; m <<= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

template <int L>
__device__ __forceinline__ float lanes_max(float v)
{
#pragma unroll
    for (int m = 1; m < L; m <<= 1)
        v = fmaxf(v, __shfl_xor(v, m, 64));
    return v;
}

template <int L>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t v)
{
    v = group_max<(L < 16 ? L : 16)>(v);
#pragma unroll
    for (int m = 16; m < L; m <<= 1)
        v = umax(v, (uint32_t)__shfl_xor((int)v, m, 64));
    return v;
}

// V consecutive elements of a row from element e0 on; those at or past
// `width` become `fill`.  `whole`: width is a multiple of V, so a lane's
// elements are all inside or all outside.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *row, int e0, int width, bool whole, float fill, float (&v)[V])
{
    typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    if (V > 1 && whole) {
        if (e0 < width) {
            const Vec x = *reinterpret_cast<const Vec *>(row + e0);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = Piece<T>::to_f32(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = fill;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = e0 + i < width ? Piece<T>::to_f32(row[e0 + i]) : fill;
}

// Workspace of a call: per run, the counts and probability sums of every
// expert and the run's sum of lse^2 and number of live tokens.
struct RouteWorkspace {
    int32_t *counts;  // [runs][experts]
    float *probs;     // [runs][experts]
    float *z;         // [runs]
    int32_t *live;    // [runs]
};

// One run of tokens per workgroup.  L lanes per token, V experts per lane.
template <typename T, int L, int V, int THREADS>
__global__ __launch_bounds__(THREADS) void moe_route_kernel(
    const T *__restrict__ logits, int64_t sl, int tokens, int experts, const uint8_t *__restrict__ mask, int k,
    int renorm, int run, int32_t *__restrict__ ids, float *__restrict__ weights, int32_t *__restrict__ rows,
    float *__restrict__ lse_out, RouteWorkspace ws)
{
    constexpr int G = THREADS / L;  // tokens in flight
    constexpr int WAVES = THREADS / 64;
    // per expert the 64-token mask and the run's count so far; per slot of the
    // round its probability and expert, per token 1 / (sum of its slots)
    extern __shared__ uint64_t lds[];
    uint64_t *bits = lds;
    int32_t *count = reinterpret_cast<int32_t *>(bits + experts);
    float *norm = reinterpret_cast<float *>(count + experts);
    float *slot_p = norm + kRouteTile;
    uint16_t *slot_e = reinterpret_cast<uint16_t *>(slot_p + kRouteTile * k);
    const int tid = threadIdx.x, sub = tid % L, grp = tid / L;
    const int e0 = sub * V;
    const bool whole = experts % V == 0;
    for (int e = tid; e < experts; e += THREADS) {
        bits[e] = 0;
        count[e] = 0;
    }
    float acc[V], zsum = 0.0f;
    int nlive = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.0f;
    __syncthreads();
    const int first = blockIdx.x * run, last = min(first + run, tokens);
    for (int t0 = first; t0 < last; t0 += kRouteTile) {
        for (int s = grp; s < kRouteTile; s += G) {
            const int t = t0 + s;
            const bool in = t < last;
            float v[V];
            const int tl = in ? t : first;
            load_row<T, V>(logits + (int64_t)tl * sl, e0, experts, whole, -INFINITY, v);
            bool live = in && (!mask || mask[tl] != 0);
            float top = v[0];
            bool bad = false;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                top = fmaxf(top, v[i]);
                bad |= v[i] != v[i];
            }
            top = lanes_max<L>(top);
            // fmax drops NaN: a row of -inf and NaN alone has no logit either
            live = live && top > -INFINITY;
            float p[V], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = __expf(v[i] - top);
                sum += p[i];
            }
            sum = lanes_sum<L>(sum);
            const float lse = live ? logf(sum) + top : INFINITY;
            const float inv = 1.0f / sum;
            if (live) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] += p[i] * inv;
                if (sub == 0) {
                    zsum = fmaf(lse, lse, zsum);
                    ++nlive;
                }
            }
            if (in && sub == 0)
                lse_out[t] = lse;
            // the k largest: a lane offers its best, the largest offer wins,
            // the lowest lane among equals (its experts come first)
            uint32_t key[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = live ? route_key(v[i]) : 0u;
            float total = 0.0f;
            for (int j = 0; j < k; ++j) {
                uint32_t best = 0;
                int at = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] > best) {
                        best = key[i];
                        at = i;
                    }
                const uint32_t win = lanes_umax<L>(best);
                const uint64_t same = __ballot(best == win) >> ((tid & 63) / L * L);
                const bool owner = sub == __builtin_ctzll(same);
                if (owner) {
                    float pw = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i == at) {
                            pw = p[i] * inv;
                            key[i] = 0;
                        }
                    const bool taken = win != 0;
                    slot_p[s * k + j] = taken ? pw : 0.0f;
                    slot_e[s * k + j] = taken ? (uint16_t)(e0 + at) : kNoExpert;
                    if (taken) {
                        atomicOr(reinterpret_cast<unsigned long long *>(bits + e0 + at), 1ull << s);
                        total += pw;
                    }
                }
            }
            total = lanes_sum<L>(total);
            if (sub == 0)
                norm[s] = renorm && total > 0.0f ? 1.0f / total : 1.0f;
        }
        __syncthreads();
        // rank of each slot among the run's slots of its expert
        const int n = min(kRouteTile, last - t0) * k;
        for (int i = tid; i < n; i += THREADS) {
            const int s = i / k;
            const int64_t at = (int64_t)t0 * k + i;
            const int e = slot_e[i];
            const bool taken = e != kNoExpert;
            ids[at] = taken ? e : -1;
            weights[at] = slot_p[i] * norm[s];
            rows[at] = taken ? count[e] + __popcll(bits[e] & ((1ull << s) - 1)) : -1;
        }
        __syncthreads();
        for (int e = tid; e < experts; e += THREADS) {
            count[e] += __popcll(bits[e]);
            bits[e] = 0;
        }
        __syncthreads();
    }
    // the run's sums, wave after wave so that their order is fixed
    float *psum = reinterpret_cast<float *>(bits);
    const int wave = tid >> 6, lane = tid & 63;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int m = L; m < 64; m <<= 1)
            acc[i] += __shfl_xor(acc[i], m, 64);
    zsum = lanes_sum<64>(zsum);
    nlive = (int)lanes_sum<64>((float)nlive);
    if (lane == 0) {
        norm[wave] = zsum;
        norm[WAVES + wave] = (float)nlive;
    }
    for (int w = 0; w < WAVES; ++w) {
        if (wave == w && lane < L)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < experts)
                    psum[e0 + i] = (w ? psum[e0 + i] : 0.0f) + acc[i];
        __syncthreads();
    }
    for (int e = tid; e < experts; e += THREADS) {
        ws.counts[(int64_t)blockIdx.x * experts + e] = count[e];
        ws.probs[(int64_t)blockIdx.x * experts + e] = psum[e];
    }
    if (tid == 0) {
        float z = 0.0f, n = 0.0f;
        for (int w = 0; w < WAVES; ++w) {
            z += norm[w];
            n += norm[WAVES + w];
        }
        ws.z[blockIdx.x] = z;
        ws.live[blockIdx.x] = (int)n;
    }
}

// sum over the workgroup's kRankThreads values in a fixed order
__device__ __forceinline__ double tree_sum(double *part, double v)
{
    const int tid = threadIdx.x;
    part[tid] = v;
    __syncthreads();
    for (int m = kRankThreads / 2; m > 0; m >>= 1) {
        if (tid < m)
            part[tid] += part[tid + m];
        __syncthreads();
    }
    const double s = part[0];
    __syncthreads();
    return s;
}

// Ranks over all tokens.  Workgroup b < gridDim.x - 1 takes the slots of
// `group` runs; the last one writes the per-expert results.  Every workgroup
// adds up the runs' counts itself (they are small and in cache), each expert
// by several threads, then lays the groups out.
__global__ __launch_bounds__(kRankThreads) void moe_rank_kernel(
    int tokens, int experts, int k, int align, int run, int nruns, int group, const int32_t *__restrict__ ids,
    int32_t *__restrict__ rows, int32_t *__restrict__ counts, int32_t *__restrict__ offs,
    float *__restrict__ mean_prob, float *__restrict__ losses, int32_t *__restrict__ live, RouteWorkspace ws)
{
    extern __shared__ uint64_t lds[];
    int32_t *total = reinterpret_cast<int32_t *>(lds);    // [experts] counts, then group starts
    int32_t *before = total + experts;                     // [experts] in the runs before this workgroup's
    const int tid = threadIdx.x;
    const bool final = blockIdx.x == gridDim.x - 1;
    const int run0 = blockIdx.x * group, run1 = min(run0 + group, nruns);
    for (int e = tid; e < 2 * experts; e += kRankThreads)
        total[e] = 0;
    __syncthreads();
    // integer sums: their order does not matter
    const int parts = max(1, kRankThreads / experts);
    for (int i = tid; i < parts * experts; i += kRankThreads) {
        const int e = i % experts, part = i / experts;
        int all = 0, prior = 0;
#pragma unroll 8
        for (int r = part; r < nruns; r += parts) {
            const int c = ws.counts[(int64_t)r * experts + e];
            all += c;
            prior += r < run0 ? c : 0;
        }
        atomicAdd(&total[e], all);
        if (!final)
            atomicAdd(&before[e], prior);
    }
    __syncthreads();
    if (final) {
        // per-expert results, and the losses in 64 bits in a fixed order
        __shared__ double part[kRankThreads];
        __shared__ int alive;
        if (tid == 0)
            alive = 0;
        __syncthreads();
        if (tid < nruns)
            atomicAdd(&alive, ws.live[tid]);
        const double z = tree_sum(part, tid < nruns ? (double)ws.z[tid] : 0.0);
        const int n = alive;
        const double inv = n > 0 ? 1.0 / (double)n : 0.0;
        double s = 0.0;
        for (int e = tid; e < experts; e += kRankThreads) {
            double p = 0.0;
#pragma unroll 8
            for (int r = 0; r < nruns; ++r)
                p += (double)ws.probs[(int64_t)r * experts + e];
            p *= inv;
            mean_prob[e] = (float)p;
            counts[e] = total[e];
            s += (double)total[e] * p;
        }
        s = tree_sum(part, s);
        if (tid == 0) {
            losses[0] = (float)(s * (double)experts * inv / (double)k);
            losses[1] = (float)(z * inv);
            live[0] = n;
        }
    }
    // group starts: wave 0 scans 64 experts at a time
    if (tid < 64) {
        int base = 0;
        for (int e0 = 0; e0 < experts; e0 += 64) {
            const int e = e0 + tid;
            const int c = e < experts ? total[e] : 0;
            const int padded = (c + align - 1) / align * align;
            int sum = padded;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int up = __shfl_up(sum, m, 64);
                sum += tid >= m ? up : 0;
            }
            if (e < experts) {
                if (final)
                    offs[e] = base + sum;
                total[e] = base + sum - padded;
            }
            base += __shfl(sum, 63, 64);
        }
    }
    __syncthreads();
    if (final)
        return;
    for (int r = run0; r < run1; ++r) {
        const int64_t first = (int64_t)r * run * k, last = min((int64_t)(r + 1) * run, (int64_t)tokens) * k;
        for (int64_t i = first + tid; i < last; i += kRankThreads) {
            const int e = ids[i];
            if (e >= 0)
                rows[i] += total[e] + before[e];
        }
        __syncthreads();
        for (int e = tid; e < experts; e += kRankThreads)
            before[e] += ws.counts[(int64_t)r * experts + e];
        __syncthreads();
    }
}

// dl_te = p_te (g_te - sum_e' p_te' g_te') + 2 g_z lse_t p_te / n with
// g_te = g_b E c_e / (n^2 k) + [e = ids_tj] q_tj, where q is the gradient of
// the selected probabilities (through the renormalisation when there is one).
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(
    const T *__restrict__ logits, int64_t sl, int tokens, int experts, int k, int renorm,
    const int32_t *__restrict__ ids, const float *__restrict__ weights, const float *__restrict__ lse_in,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ live, const float *__restrict__ gw,
    const float *__restrict__ gl, T *__restrict__ dl, int64_t sd)
{
    const int tid = threadIdx.x, sub = tid % L, e0 = sub * V;
    const bool whole = experts % V == 0;
    const float n = (float)max(live ? live[0] : 1, 1);
    const float gb = gl ? gl[0] * (float)experts / (n * (float)k) / n : 0.0f;
    const float gz = gl ? 2.0f * gl[1] / n : 0.0f;
    float bal[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        bal[i] = gl && e0 + i < experts ? gb * (float)counts[e0 + i] : 0.0f;
    const int64_t per_grid = (int64_t)gridDim.x * (256 / L);
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + tid / L; t < tokens; t += per_grid) {
        float v[V];
        load_row<T, V>(logits + t * sl, e0, experts, whole, -INFINITY, v);
        const float lse = lse_in[t];
        const bool dead = lse == INFINITY;
        float p[V], g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = dead || v[i] == -INFINITY ? 0.0f : __expf(v[i] - lse);
            g[i] = bal[i];
        }
        if (gw) {
            float total = 1.0f, wg = 0.0f;
            if (renorm) {
                total = 0.0f;
                for (int j = 0; j < k; ++j) {
                    const int e = ids[t * k + j];
                    if (e >= 0)
                        wg = fmaf(weights[t * k + j], gw[t * k + j], wg);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        total += e == e0 + i ? p[i] : 0.0f;
                }
                total = lanes_sum<L>(total);
            }
            const float inv = 1.0f / total;
            for (int j = 0; j < k; ++j) {
                const int e = ids[t * k + j];
                const float q = (gw[t * k + j] - wg) * inv;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    g[i] += e == e0 + i ? q : 0.0f;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            dot = fmaf(p[i], g[i], dot);
        dot = lanes_sum<L>(dot) - gz * lse;
        typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
        T *out = dl + t * sd + e0;
        Vec o;
#pragma unroll
        for (int i = 0; i < V; ++i)
            o[i] = Piece<T>::from_f32(dead ? 0.0f : p[i] * (g[i] - dot));
        if (whole) {
            if (e0 < experts)
                *reinterpret_cast<Vec *>(out) = o;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < experts)
                    out[i] = o[i];
        }
    }
}

}  // namespace mxq
