// A whole mixture-of-experts layer for a few tokens: what a serving step runs.
//
//   ids_t, s_t = the top_k experts of token t and their softmax weights
//   h_tj = s_tj act(U_e x_t + a_e)            e = ids_tj; gated: act(gate) * value
//   y_t  = resid_t + sum_j (D_e h_tj + s_tj b_e)
//
// Everything is bound by the active experts' weights, read once each: few
// tokens share them.  Both products put 16 rows of weights against 16 tokens on
// a matrix instruction that would take as long for one token, weights straight
// from memory into registers, so what a wave does is load.
//   up    a workgroup per active expert and 32 rows of U; its waves take the
//         parts of the sum
//   down  the sum over experts and over h is one long sum: a workgroup per 16
//         rows of D, its waves (and, for few rows, several workgroups) take the
//         parts; a token that does not use an expert has zeros there
// h passes in two bf16 parts (16 bits): the second costs matrix instructions,
// of which there are plenty, not weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_ops.hpp"
#include "stream_ops.hpp"
#include "mxq_device.hpp"
#include "tile_ops.hpp"
#include "wave_ops.hpp"

namespace mxq {

constexpr int kLayerTokens = 64, kLayerExperts = 1024, kLayerThreads = 256;
constexpr int kUnit = 256;   // values of the down product's sum that a wave takes at a time

struct LayerWeights {
    const void *w;           // (experts, rows, cols) bf16 or e4m3, elements along cols
    int64_t se, sr;
    const uint8_t *scales;   // e8m0, blocks along cols
    int64_t sse, ssr;
    const void *bias;
    int64_t sb;
    int bias_f32;
};

struct LayerArgs {
    const uint16_t *x;
    int64_t sx;
    const void *logits;
    int64_t sl;
    const uint8_t *mask;
    int tokens, width, hidden, experts, k, renorm, act;
    LayerWeights up, down;
    const uint16_t *resid;
    int64_t sr;
    uint16_t *y;
    int64_t sy;
    int32_t *ids;            // workspace: (tokens, k)
    float *share;            // (tokens, k)
    uint16_t *hi, *lo;       // (tokens * k, hp)
    int hp;
    float *parts;            // (splits, tokens, width)
    int splits;
};

// ---------------------------------------------------------------- selection

// One wave per token.  Lane l holds experts l V .. l V + V - 1, so that among
// equal logits the first lane, and in it the first value, has the lowest
// expert.  -inf and NaN are never taken.
template <typename T, int V>
__device__ __forceinline__ void select_token(const LayerArgs &a, int t, int32_t *ids, float *share)
{
    const int lane = threadIdx.x & 63;
    const T *row = reinterpret_cast<const T *>(a.logits) + t * a.sl;
    float x[V];
    uint32_t key[V];
    const bool live = !a.mask || a.mask[t];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        x[v] = e < a.experts ? Piece<T>::to_f32(row[e]) + 0.0f : -INFINITY;  // one zero
        const uint32_t b = __float_as_uint(x[v]);
        key[v] = live && x[v] > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
    }
    int id = -1;
    float top = 0.0f, sum = 0.0f, own = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            best = umax(best, key[v]);
        const uint32_t most = wave_max(best);
        if (most == 0)
            break;
        const int from = __builtin_ctzll(__ballot(best == most));
        int at = 0;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            at = key[v] == most ? v : at;
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = lane == from && v == at ? 0u : key[v];
        const int e = __builtin_amdgcn_readlane(lane * V + at, from);
        const float l = __uint_as_float(most & 0x80000000u ? most & 0x7fffffffu : ~most);
        top = j == 0 ? l : top;
        const float ex = __expf(l - top);
        sum += ex;
        id = lane == j ? e : id;
        own = lane == j ? ex : own;
    }
    // the sum over all experts: a NaN among them makes the token's weights NaN
    float all = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        all += lane * V + v < a.experts ? __expf(x[v] - top) : 0.0f;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        all += __shfl_xor(all, m, 64);
    if (lane < a.k) {
        ids[t * a.k + lane] = id;
        share[t * a.k + lane] = id < 0 ? 0.0f : all == all ? own / (a.renorm ? sum : all) : all;
    }
}

template <typename T>
__device__ __forceinline__ void select_tokens(const LayerArgs &a, int first, int step, int32_t *ids, float *share)
{
    for (int t = first; t < a.tokens; t += step) {
        if (a.experts <= 64)
            select_token<T, 1>(a, t, ids, share);
        else if (a.experts <= 256)
            select_token<T, 4>(a, t, ids, share);
        else
            select_token<T, 16>(a, t, ids, share);
    }
}

template <typename T>
__global__ __launch_bounds__(64) void layer_select_kernel(LayerArgs a)
{
    select_tokens<T>(a, blockIdx.x, gridDim.x, a.ids, a.share);
}

// The experts that some slot names, as a bit per expert; ends with a barrier.
__device__ __forceinline__ void active_bits(const LayerArgs &a, const int32_t *ids, uint32_t *bits)
{
    for (int i = threadIdx.x; i < kLayerExperts / 32; i += kLayerThreads)
        bits[i] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.tokens * a.k; s += kLayerThreads)
        if (ids[s] >= 0)
            atomicOr(&bits[ids[s] >> 5], 1u << (ids[s] & 31));
    __syncthreads();
}

// Bits set before word lane (lanes 0..31), and in all.
__device__ __forceinline__ int bits_before(const uint32_t *bits, int &total)
{
    const int lane = threadIdx.x & 63, n = lane < kLayerExperts / 32 ? __popc(bits[lane]) : 0, upto = wave_scan(n);
    total = __builtin_amdgcn_readlane(upto, 63);
    return upto - n;
}

// ---------------------------------------------------------------- up

// acc[i][f] += rows i of weights times tokens f over [k0, k1) of the sum
template <bool MX, int FT, int U>
__device__ __forceinline__ void up_range(const void *const (&row)[2], const uint8_t *const (&scales)[2], const uint16_t *const (&x)[FT],
                                         const bool (&there)[FT], int k0, int k1, int end, float4v (&acc)[2][FT])
{
    typedef WeightStep<MX> Step;
    int k = k0;
    for (; k + U * Step::K <= k1; k += U * Step::K) {
        Step s[2][U];
        bf16x8 t[FT][U][Step::PIECES];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s[i][u].load(row[i], scales[i], k + u * Step::K);
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int h = 0; h < Step::PIECES; ++h)
                    t[f][u][h] = there[f] ? token_piece<MX>(x[f], k + u * Step::K, h) : zero_piece();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < Step::PIECES; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int f = 0; f < FT; ++f)
                        acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[i][u].piece(h), t[f][u][h], acc[i][f], 0, 0, 0);
    }
    for (; k < k1; k += Step::K) {
        Step s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            s[i].load_tail(row[i], scales[i], k, end);
#pragma unroll
        for (int h = 0; h < Step::PIECES; ++h)
#pragma unroll
            for (int f = 0; f < FT; ++f) {
                const bf16x8 t = there[f] ? token_piece_tail<MX>(x[f], k, h, end) : zero_piece();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[i].piece(h), t, acc[i][f], 0, 0, 0);
            }
    }
}

// list: the expert's slots; the four waves' sums meet in `sums`
template <bool MX, bool GATED, int FT>
__device__ __forceinline__ void up_tokens(const LayerArgs &a, int e, int r0, const int16_t *list, int count,
                                          const float *share, float4v *sums)
{
    typedef WeightStep<MX> Step;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), fr = lane & 15;
    const int wide = GATED ? 2 * a.hidden : a.hidden;
    const void *row[2];
    const uint8_t *scales[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // rows past the last: the last one's, whose results are dropped
        const int r = GATED ? min(r0 + fr, a.hidden - 1) + i * a.hidden : min(r0 + i * 16 + fr, wide - 1);
        row[i] = reinterpret_cast<const char *>(a.up.w) + (e * a.up.se + r * a.up.sr) * (MX ? 1 : 2);
        scales[i] = MX ? a.up.scales + e * a.up.sse + r * a.up.ssr : nullptr;
    }
    const uint16_t *x[FT];
    bool there[FT];
#pragma unroll
    for (int f = 0; f < FT; ++f) {
        there[f] = f * 16 + fr < count;
        x[f] = a.x + (there[f] ? list[f * 16 + fr] / a.k : 0) * a.sx;
    }
    float4v acc[2][FT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int f = 0; f < FT; ++f)
            acc[i][f] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (a.width + Step::K - 1) / Step::K;
    up_range<MX, FT, FT == 1 ? 8 / Step::PIECES : 4 / Step::PIECES>(
        row, scales, x, there, steps * wave / 4 * Step::K, min(steps * (wave + 1) / 4 * Step::K, a.width), a.width, acc);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int f = 0; f < FT; ++f)
            sums[((wave * 2 + i) * FT + f) * 64 + lane] = acc[i][f];
    __syncthreads();
    // a lane has four rows of a token; gated: of gate and value both
    constexpr int ITEMS = GATED ? FT : 2 * FT;
    for (int at = threadIdx.x; at < ITEMS * 64; at += kLayerThreads) {
        const int i = at / (FT * 64), f = at / 64 % FT, l = at & 63, token = f * 16 + (l & 15);
        if (token >= count)
            continue;
        float4v z[2];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            z[h] = sums[((GATED ? h : i) * FT + f) * 64 + l];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                z[h] += sums[((w * 2 + (GATED ? h : i)) * FT + f) * 64 + l];
        }
        const int slot = list[token];
        const float s = share[slot];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = r0 + (GATED ? 0 : i * 16) + 4 * (l >> 4) + q;
            if (r >= a.hidden)
                continue;
            float v = z[0][q];
            if (a.up.bias)
                v += bias_at(a.up.bias, a.up.bias_f32, e * a.up.sb + r);
            v = act_value(a.act, v);
            if constexpr (GATED) {
                float g = z[1][q];
                if (a.up.bias)
                    g += bias_at(a.up.bias, a.up.bias_f32, e * a.up.sb + a.hidden + r);
                v *= g;
            }
            v *= s;
            const uint16_t hi = Piece<uint16_t>::from_f32(v);
            a.hi[(int64_t)slot * a.hp + r] = hi;
            const float rest = v - Piece<uint16_t>::to_f32(hi);  // of an infinity: NaN
            a.lo[(int64_t)slot * a.hp + r] = Piece<uint16_t>::from_f32(fabsf(rest) < INFINITY ? rest : 0.0f);
        }
    }
}

// LDS: ids, shares, then the waves' sums.  FT: fragments of 16 tokens that an
// expert can have (a call of at most 16 tokens has registers for one alone)
template <typename T, bool MX, bool GATED, int FT, bool SELECT>
__global__ __launch_bounds__(kLayerThreads) void layer_up_kernel(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ uint32_t bits[kLayerExperts / 32];
    __shared__ int16_t list[kLayerTokens];
    __shared__ int found[2];
    const int slots = a.tokens * a.k, wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int32_t *ids = reinterpret_cast<int32_t *>(lds);
    float *share = reinterpret_cast<float *>(ids + slots);
    float4v *sums = reinterpret_cast<float4v *>(lds + ((slots * 8 + 15) & ~15));
    if constexpr (SELECT) {
        select_tokens<T>(a, wave, kLayerThreads / 64, ids, share);
        __syncthreads();
        if (blockIdx.x == 0 && blockIdx.y == 0)
            for (int s = threadIdx.x; s < slots; s += kLayerThreads) {
                a.ids[s] = ids[s];
                a.share[s] = share[s];
            }
    } else {
        for (int s = threadIdx.x; s < slots; s += kLayerThreads) {
            ids[s] = a.ids[s];
            share[s] = a.share[s];
        }
        __syncthreads();
    }
    active_bits(a, ids, bits);
    if (wave == 0) {
        // active expert number blockIdx.y, and its slots in order
        int total;
        const int before = bits_before(bits, total), n = (int)blockIdx.y;
        const uint64_t reached = __ballot(lane < kLayerExperts / 32 && before <= n);
        const int word = 63 - __builtin_clzll(reached);
        uint32_t left = bits[word];
        for (int i = __builtin_amdgcn_readlane(before, word); i < n && left; ++i)
            left &= left - 1;
        const int e = n < total ? word * 32 + __builtin_ctz(left) : -1;
        int count = 0;
        for (int s0 = 0; s0 < slots; s0 += 64) {
            const bool mine = s0 + lane < slots && e >= 0 && ids[s0 + lane] == e;
            const uint64_t m = __ballot(mine);
            const int at = count + __popcll(m & ((1ull << lane) - 1));
            if (mine && at < kLayerTokens)
                list[at] = (int16_t)(s0 + lane);
            count += __popcll(m);
        }
        if (lane == 0) {
            found[0] = e;
            found[1] = min(count, kLayerTokens);
        }
    }
    __syncthreads();
    const int e = uniform(found[0]), count = uniform(found[1]);
    if (e < 0)
        return;
    const int r0 = blockIdx.x * (GATED ? 16 : 32);
    if (FT == 1 || count <= 16)
        up_tokens<MX, GATED, 1>(a, e, r0, list, count, share, sums);
    else if (count <= 32)
        up_tokens<MX, GATED, 2>(a, e, r0, list, count, share, sums);
    else
        up_tokens<MX, GATED, 4>(a, e, r0, list, count, share, sums);
}

// ---------------------------------------------------------------- down

// y's values of four rows of one token from the finished sums
__device__ __forceinline__ void layer_result(const LayerArgs &a, int t, int d, float v)
{
    if (a.down.bias)
        for (int j = 0; j < a.k; ++j) {
            const int e = a.ids[t * a.k + j];
            if (e >= 0)
                v += a.share[t * a.k + j] * bias_at(a.down.bias, a.down.bias_f32, e * a.down.sb + d);
        }
    if (a.resid)
        v += Piece<uint16_t>::to_f32(a.resid[t * a.sr + d]);
    a.y[t * a.sy + d] = Piece<uint16_t>::from_f32(v);
}

// LDS: the active experts, where each expert stands among them, each (active
// expert, token)'s slot
template <bool MX, int FT>
__global__ __launch_bounds__(kLayerThreads) void layer_down_kernel(LayerArgs a, int most)
{
    typedef WeightStep<MX> Step;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ uint32_t bits[kLayerExperts / 32];
    __shared__ float4v sums[kLayerThreads / 64][FT][64];
    int16_t *active = reinterpret_cast<int16_t *>(lds);
    int16_t *place = active + most;
    uint8_t *slot_of = reinterpret_cast<uint8_t *>(place + a.experts);
    const int slots = a.tokens * a.k, wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, fr = lane & 15;
    active_bits(a, a.ids, bits);
    for (int i = threadIdx.x; i < most * a.tokens; i += kLayerThreads)
        slot_of[i] = 0xff;
    int total;
    {
        const int before = bits_before(bits, total);
        if (wave == 0 && lane < kLayerExperts / 32) {
            int at = before;
            for (uint32_t left = bits[lane]; left; left &= left - 1, ++at) {
                const int e = lane * 32 + __builtin_ctz(left);
                active[at] = (int16_t)e;
                place[e] = (int16_t)at;
            }
        }
    }
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += kLayerThreads)
        if (a.ids[s] >= 0)
            slot_of[place[a.ids[s]] * a.tokens + s / a.k] = (uint8_t)(s % a.k);
    __syncthreads();

    const int d0 = blockIdx.x * 16, r = min(d0 + fr, a.width - 1);
    const int per = (a.hidden + kUnit - 1) / kUnit, units = total * per;
    const int parts = a.splits * 4, own = blockIdx.y * 4 + wave;
    const int u1 = (int)((int64_t)units * (own + 1) / parts);
    float4v acc[FT];
#pragma unroll
    for (int f = 0; f < FT; ++f)
        acc[f] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = (int)((int64_t)units * own / parts); u < u1; ++u) {
        const int n = u / per, k0 = u % per * kUnit, e = uniform(active[n]);
        const char *row = reinterpret_cast<const char *>(a.down.w) + (e * a.down.se + r * a.down.sr) * (MX ? 1 : 2);
        const uint8_t *scales = MX ? a.down.scales + e * a.down.sse + r * a.down.ssr : nullptr;
        constexpr int STEPS = kUnit / Step::K;
        Step s[STEPS];
        const bool whole = k0 + kUnit <= a.hidden;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (whole)
                s[i].load(row, scales, k0 + i * Step::K);
            else
                s[i].load_tail(row, scales, k0 + i * Step::K, a.hidden);
        }
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            const int t = f * 16 + fr, j = t < a.tokens ? slot_of[n * a.tokens + t] : 0xff;
            const bool there = j != 0xff;
            if (!__ballot(there))
                continue;
            const int64_t at = there ? (int64_t)(t * a.k + j) * a.hp : 0;
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int h = 0; h < Step::PIECES; ++h) {
                    const int k = k0 + i * Step::K;
                    if (!whole && k >= a.hidden)
                        continue;
                    bf16x8 hi = zero_piece(), lo = zero_piece();
                    if (there) {
                        hi = whole ? token_piece<MX>(a.hi + at, k, h) : token_piece_tail<MX>(a.hi + at, k, h, a.hidden);
                        lo = whole ? token_piece<MX>(a.lo + at, k, h) : token_piece_tail<MX>(a.lo + at, k, h, a.hidden);
                    }
                    const bf16x8 w = s[i].piece(h);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, lo, acc[f], 0, 0, 0);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, hi, acc[f], 0, 0, 0);
                }
        }
    }
#pragma unroll
    for (int f = 0; f < FT; ++f)
        sums[wave][f][lane] = acc[f];
    __syncthreads();
    for (int at = threadIdx.x; at < FT * 64; at += kLayerThreads) {
        const int f = at / 64, l = at & 63, t = f * 16 + (l & 15);
        if (t >= a.tokens)
            continue;
        const float4v v = (sums[0][f][l] + sums[1][f][l]) + (sums[2][f][l] + sums[3][f][l]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = d0 + 4 * (l >> 4) + q;
            if (d >= a.width)
                continue;
            if (a.splits > 1)
                a.parts[((int64_t)blockIdx.y * a.tokens + t) * a.width + d] = v[q];
            else
                layer_result(a, t, d, v[q]);
        }
    }
}

// the parts of the down product's sums, in order
__global__ __launch_bounds__(kLayerThreads) void layer_join_kernel(LayerArgs a)
{
    const int d = blockIdx.x * kLayerThreads + threadIdx.x, t = blockIdx.y;
    if (d >= a.width)
        return;
    float v = 0.0f;
    for (int s = 0; s < a.splits; ++s)
        v += a.parts[((int64_t)s * a.tokens + t) * a.width + d];
    layer_result(a, t, d, v);
}

}  // namespace mxq
