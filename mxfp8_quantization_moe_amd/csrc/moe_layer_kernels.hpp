// A whole mixture-of-experts layer for a few tokens: what a serving step runs.
//
//   ids_t, s_t = the top_k experts of token t and their softmax weights
//   h_tj = s_tj act(U_e x_t + a_e)            e = ids_tj; gated: act(gate) * value
//   y_t  = resid_t + sum_j (D_e h_tj + s_tj b_e)
//
// Everything is bound by the active experts' weights, read once each: few
// tokens share them.  Both products put 16 rows of weights against up to 16
// tokens on a matrix instruction that would take as long for one token, weights
// straight from memory into registers, so what a wave does is load.
//   select  one workgroup: the tokens' experts, and the slots in the order of
//           their experts (one token alone selects within the up kernel)
//   up      a workgroup per active expert and 16 or 32 rows of U; its waves take
//           the parts of the sum
//   down    the sum over experts and over h is one long sum: a workgroup per 8
//           rows of D, its waves (and, for few rows, several workgroups) take the
//           parts and gather the tokens' sums in LDS.  Eight rows fill the
//           instruction's 16 with the two halves of the sum, against 8 tokens in
//           two halves; twice the workgroups of 16 rows, enough for the chip
//           without a pass that joins them from 2048 rows on
// h passes in two bf16 parts (16 bits): the second costs matrix instructions,
// of which there are plenty, not weights.
//
// us, per kernel:                              select    up        down
//   1 token, 8 of 256 experts of 2048 x 768       -      14.7       9.5
//   8 tokens, the same in MXFP8 (280 MB)          5.8    48 (3.9)   32 (2.9 TB/s)
//   64 tokens, 4 of 128 experts of 4096 x 1024   14.8   272 (6.6)  208 (4.3)
//   5 tokens, 3 of 13 experts of 1111 x 333       3.9     9.8      12.2
// Few experts end after one or two latencies of memory; many are bound by it,
// in the down product also by the slots' sums, which meet in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "linear_ops.hpp"
#include "stream_ops.hpp"
#include "mxq_device.hpp"
#include "tile_ops.hpp"
#include "wave_ops.hpp"

namespace mxq {

constexpr int kLayerTokens = 64, kLayerSlots = 32, kLayerExperts = 1024, kLayerThreads = 256;
constexpr int kSelectThreads = 1024, kDownWaves = 16, kDownWavesMx = 12;

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
    int32_t *active;         // experts that some slot names
    int32_t *begin;          // (active + 1) where their slots begin; [most + 1]: how many they are
    int32_t *order;          // slots, expert after expert
    int most;                // active experts at most
    uint16_t *hi, *lo;       // (tokens * k, hp)
    int hp;
    float *parts;            // (splits, tokens, width)
    int splits;
};

// ---------------------------------------------------------------- selection

// A wave selects for tokens first, first + step, ... below `tokens`, NT at a
// time, whose chains of reductions overlap.  Lane l holds experts l V .. l V +
// V - 1, so that among equal logits the first lane, and in it the first value,
// has the lowest expert.  -inf and NaN are never taken.
template <typename T, int V, int NT>
__device__ __forceinline__ void select_wave(const LayerArgs &a, int first, int step, int32_t *ids, float *share)
{
    const int lane = threadIdx.x & 63;
    for (int t0 = first; t0 < a.tokens; t0 += NT * step) {
        float x[NT][V], top[NT], sum[NT], own[NT];
        uint32_t key[NT][V];
        int id[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = min(t0 + i * step, a.tokens - 1);
            const T *row = reinterpret_cast<const T *>(a.logits) + t * a.sl;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane * V + v;
                x[i][v] = e < a.experts ? Piece<T>::to_f32(row[e]) + 0.0f : -INFINITY;  // one zero
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const bool live = !a.mask || a.mask[min(t0 + i * step, a.tokens - 1)];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t b = __float_as_uint(x[i][v]);
                key[i][v] = live && x[i][v] > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
            }
            id[i] = -1;
            top[i] = sum[i] = own[i] = 0.0f;
        }
        for (int j = 0; j < a.k; ++j) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                uint32_t best = key[i][0];
#pragma unroll
                for (int v = 1; v < V; ++v)
                    best = umax(best, key[i][v]);
                const uint32_t most = wave_max(best);
                // none left: lane 0 takes its first value, which is dropped
                const int from = __builtin_ctzll(__ballot(best == most));
                int at = 0;
#pragma unroll
                for (int v = V - 1; v >= 0; --v)
                    at = key[i][v] == most ? v : at;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    key[i][v] = lane == from && v == at ? 0u : key[i][v];
                const int e = most ? __builtin_amdgcn_readlane(lane * V + at, from) : -1;
                const float l = __uint_as_float(most & 0x80000000u ? most & 0x7fffffffu : ~most);
                top[i] = j == 0 && most ? l : top[i];
                const float ex = most ? __expf(l - top[i]) : 0.0f;
                sum[i] += ex;
                id[i] = lane == j ? e : id[i];
                own[i] = lane == j ? ex : own[i];
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            // the sum over all experts: a NaN among them makes the token's weights NaN
            float all = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                all += lane * V + v < a.experts ? __expf(x[i][v] - top[i]) : 0.0f;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1)
                all += __shfl_xor(all, m, 64);
            const int t = t0 + i * step;
            if (t < a.tokens && lane < a.k) {
                ids[t * a.k + lane] = id[i];
                share[t * a.k + lane] = id[i] < 0 ? 0.0f : all == all ? own[i] / (a.renorm ? sum[i] : all) : all;
            }
        }
    }
}

template <typename T, int NT>
__device__ __forceinline__ void select_tokens(const LayerArgs &a, int first, int step, int32_t *ids, float *share)
{
    if (a.experts <= 64)
        select_wave<T, 1, NT>(a, first, step, ids, share);
    else if (a.experts <= 256)
        select_wave<T, 4, NT>(a, first, step, ids, share);
    else
        select_wave<T, 16, (NT + 1) / 2>(a, first, step, ids, share);
}

// What the other kernels need to find their slots.  An expert's slots are in
// the order of their tokens, a token naming it at most once: the down product
// takes an expert's first 8 slots otherwise than the rest, so another order would
// round otherwise.
template <typename T>
__global__ __launch_bounds__(kSelectThreads) void layer_select_kernel(LayerArgs a)
{
    static_assert(kLayerTokens == 64 && kSelectThreads == kLayerExperts, "a bit a token, a thread an expert");
    __shared__ unsigned long long tokens[kLayerExperts];
    __shared__ int begin[kLayerExperts], sums[kSelectThreads / 64], ids[kLayerTokens * kLayerSlots];
    __shared__ float share[kLayerTokens * kLayerSlots];
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, slots = a.tokens * a.k;
    tokens[tid] = 0;
    if (a.tokens > kSelectThreads / 64)
        select_tokens<T, 4>(a, wave, kSelectThreads / 64, ids, share);
    else
        select_tokens<T, 1>(a, wave, kSelectThreads / 64, ids, share);
    __syncthreads();
    for (int s = tid; s < slots; s += kSelectThreads) {
        a.ids[s] = ids[s];
        a.share[s] = share[s];
        if (ids[s] >= 0)
            atomicOr(&tokens[ids[s]], 1ull << s / a.k);
    }
    __syncthreads();
    // expert tid: slots before its own, and its place among the active ones,
    // in the low and the high half of one sum
    const int own = __popcll(tokens[tid]), v = own | (own > 0) << 16, upto = wave_scan(v);
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    int before = upto - v, total = 0;
    for (int w = 0; w < kSelectThreads / 64; ++w) {
        if (w < wave)
            before += sums[w];
        total += sums[w];
    }
    if (own > 0) {
        a.active[before >> 16] = tid;
        a.begin[before >> 16] = before & 0xffff;
    }
    if (tid == 0) {
        a.begin[total >> 16] = total & 0xffff;
        a.begin[a.most + 1] = total >> 16;
    }
    begin[tid] = before & 0xffff;
    __syncthreads();
    for (int s = tid; s < slots; s += kSelectThreads)
        if (ids[s] >= 0)
            a.order[begin[ids[s]] + __popcll(tokens[ids[s]] & ((1ull << s / a.k) - 1))] = s;
}

// ---------------------------------------------------------------- up

// acc[i][f] += rows i of weights times tokens f over [k0, k1) of the sum
// find_tokens() sets x and there.
template <bool MX, int NF, int FT, int U, typename Find>
__device__ __forceinline__ void up_range(const void *const (&row)[NF], const uint8_t *const (&scales)[NF],
                                         const uint16_t *const (&x)[FT], const bool (&there)[FT], Find &&find_tokens,
                                         int k0, int k1, int end, float4v (&acc)[NF][FT])
{
    typedef WeightStep<MX> Step;
    struct Batch {
        Step s[NF][U];
        bf16x8 t[FT][U][Step::PIECES];
    };
    auto load_weights = [&](Batch &b, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
                b.s[i][u].load(row[i], scales[i], k + u * Step::K);
    };
    auto load_tokens = [&](Batch &b, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int h = 0; h < Step::PIECES; ++h)
                    b.t[f][u][h] = there[f] ? token_piece<MX>(x[f], k + u * Step::K, h) : zero_piece();
    };
    auto load = [&](Batch &b, int k) {
        load_weights(b, k);
        load_tokens(b, k);
    };
    auto multiply = [&](const Batch &b) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < Step::PIECES; ++h)
#pragma unroll
                for (int i = 0; i < NF; ++i)
#pragma unroll
                    for (int f = 0; f < FT; ++f)
                        acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.s[i][u].piece(h), b.t[f][u][h], acc[i][f], 0, 0, 0);
    };
    int k = k0;
    constexpr int SPAN = U * Step::K;
    if constexpr (FT == 1) {
        // the first weights go out before it is known whose tokens they meet,
        // the next loads before the products
        Batch b0, b1;
        if (k + SPAN <= k1) {
            load_weights(b0, k);
            find_tokens();
            load_tokens(b0, k);
            for (; k + 3 * SPAN <= k1; k += 2 * SPAN) {
                load(b1, k + SPAN);
                multiply(b0);
                load(b0, k + 2 * SPAN);
                multiply(b1);
            }
            if (k + 2 * SPAN <= k1) {
                load(b1, k + SPAN);
                multiply(b0);
                multiply(b1);
                k += 2 * SPAN;
            } else {
                multiply(b0);
                k += SPAN;
            }
        } else {
            find_tokens();
        }
    } else {
        find_tokens();
        Batch b;
        for (; k + SPAN <= k1; k += SPAN) {
            load(b, k);
            multiply(b);
        }
    }
    for (; k < k1; k += Step::K) {
        Step s[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i)
            s[i].load_tail(row[i], scales[i], k, end);
#pragma unroll
        for (int h = 0; h < Step::PIECES; ++h)
#pragma unroll
            for (int f = 0; f < FT; ++f) {
                const bf16x8 t = there[f] ? token_piece_tail<MX>(x[f], k, h, end) : zero_piece();
#pragma unroll
                for (int i = 0; i < NF; ++i)
                    acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[i].piece(h), t, acc[i][f], 0, 0, 0);
            }
    }
}

// Row of U that row r (0..15) of fragment i holds, from h's row r0 on.  Gated:
// of two fragments the gate's and the value's rows, of one 8 rows of either.
template <bool GATED, int NF>
__device__ __forceinline__ int up_row(int r0, int i, int r, int hidden)
{
    if (!GATED)
        return r0 + i * 16 + r;
    return NF == 2 ? r0 + r + i * hidden : r0 + (r & 7) + (r >> 3) * hidden;
}

// slot_of(c): the slot in column c < count; the four waves' sums meet in `sums`
template <bool MX, bool GATED, int NF, int FT, typename SlotOf, typename ShareOf>
__device__ __forceinline__ void up_tokens(const LayerArgs &a, int e, int r0, int count, SlotOf &&slot_of,
                                          ShareOf &&share_of, float4v *sums)
{
    typedef WeightStep<MX> Step;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), fr = lane & 15;
    const int wide = GATED ? 2 * a.hidden : a.hidden;
    const void *row[NF];
    const uint8_t *scales[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        // rows past the last: another one's, whose results are dropped
        const int r = min(up_row<GATED, NF>(r0, i, fr, a.hidden), wide - 1);
        row[i] = reinterpret_cast<const char *>(a.up.w) + (e * a.up.se + r * a.up.sr) * (MX ? 1 : 2);
        scales[i] = MX ? a.up.scales + e * a.up.sse + r * a.up.ssr : nullptr;
    }
    const uint16_t *x[FT];
    bool there[FT];
    // the item of this thread after the sums (of the first, where it has more)
    int own_slot = 0;
    float own_share = 0.0f;
    auto find_tokens = [&] {
        own_slot = slot_of(min((int)threadIdx.x % (FT * 16), count - 1));
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            there[f] = f * 16 + fr < count;
            x[f] = a.x + (there[f] ? slot_of(f * 16 + fr) / a.k : 0) * a.sx;
        }
        own_share = share_of(own_slot);
    };
    float4v acc[NF][FT];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int f = 0; f < FT; ++f)
            acc[i][f] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (a.width + Step::K - 1) / Step::K;
    up_range<MX, NF, FT, FT == 1 && MX ? 2 : 4 / (FT == 1 ? 1 : Step::PIECES)>(
        row, scales, x, there, find_tokens, steps * wave / 4 * Step::K, min(steps * (wave + 1) / 4 * Step::K, a.width), a.width, acc);
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int f = 0; f < FT; ++f)
            sums[((wave * NF + i) * FT + f) * 64 + lane] = acc[i][f];
    __syncthreads();
    auto whole = [&](int i, int f, int l) {
        float4v z = sums[(i * FT + f) * 64 + l];
#pragma unroll
        for (int w = 1; w < 4; ++w)
            z += sums[((w * NF + i) * FT + f) * 64 + l];
        return z;
    };
    // four rows of h of a token; gated: from the gate's and the value's lanes
    constexpr int ROWS = GATED ? 8 * NF : 16 * NF, ITEMS = FT * 16 * (ROWS / 4);
    for (int at = threadIdx.x; at < ITEMS; at += kLayerThreads) {
        const int c = at % (FT * 16), h0 = at / (FT * 16) * 4, f = c >> 4;
        if (c >= count)
            continue;
        float4v z, g;
        if constexpr (GATED && NF == 2) {
            z = whole(0, f, (h0 >> 2) * 16 + (c & 15));
            g = whole(1, f, (h0 >> 2) * 16 + (c & 15));
        } else if constexpr (GATED) {
            z = whole(0, f, (h0 >> 2) * 16 + (c & 15));
            g = whole(0, f, (2 + (h0 >> 2)) * 16 + (c & 15));
        } else {
            g = z = whole(h0 >> 4, f, (h0 & 15) / 4 * 16 + (c & 15));
        }
        // threads step by a multiple of the columns: the same column each time
        static_assert(kLayerThreads % (FT * 16) == 0, "own_slot is column c's");
        const int slot = own_slot;
        const float s = own_share;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = r0 + h0 + q;
            if (r >= a.hidden)
                continue;
            float v = z[q];
            if (a.up.bias)
                v += bias_at(a.up.bias, a.up.bias_f32, e * a.up.sb + r);
            v = act_value(a.act, v);
            if constexpr (GATED) {
                float w = g[q];
                if (a.up.bias)
                    w += bias_at(a.up.bias, a.up.bias_f32, e * a.up.sb + a.hidden + r);
                v *= w;
            }
            v *= s;
            const uint16_t hi = Piece<uint16_t>::from_f32(v);
            a.hi[(int64_t)slot * a.hp + r] = hi;
            const float rest = v - Piece<uint16_t>::to_f32(hi);  // of an infinity: NaN
            a.lo[(int64_t)slot * a.hp + r] = Piece<uint16_t>::from_f32(fabsf(rest) < INFINITY ? rest : 0.0f);
        }
    }
}

// FT: fragments of 16 tokens that an expert can have
template <bool MX, bool GATED, int NF, int FT>
__global__ __launch_bounds__(kLayerThreads) void layer_up_kernel(LayerArgs a)
{
    __shared__ float4v sums[4 * NF * FT * 64];
    // read together; past the active experts they are whatever was there
    const int n = (int)blockIdx.y, active = a.begin[a.most + 1], found = a.active[n], start = a.begin[n], stop = a.begin[n + 1];
    if (n >= active)
        return;
    const int e = uniform(found), first = uniform(start), count = uniform(stop) - first;
    const int r0 = blockIdx.x * (GATED ? 8 * NF : 16 * NF);
    auto slot_of = [&](int c) { return a.order[first + c]; };
    auto share_of = [&](int s) { return a.share[s]; };
    if (FT == 1 || count <= 16)
        up_tokens<MX, GATED, NF, 1>(a, e, r0, count, slot_of, share_of, sums);
    else if (FT == 2 || count <= 32)
        up_tokens<MX, GATED, NF, 2>(a, e, r0, count, slot_of, share_of, sums);
    else
        up_tokens<MX, GATED, NF, 4>(a, e, r0, count, slot_of, share_of, sums);
}

// One token: every wave selects for itself, without meeting the others; slot
// blockIdx.y is the workgroup's.  The first one leaves what the down kernel
// needs.
template <typename T, bool MX, bool GATED>
__global__ __launch_bounds__(kLayerThreads) void layer_up_one_kernel(LayerArgs a)
{
    __shared__ float4v sums[4 * 64];
    __shared__ int ids[4][kLayerSlots];
    __shared__ float share[4][kLayerSlots];
    const int wave = uniform(threadIdx.x >> 6), n = (int)blockIdx.y;
    select_tokens<T, 1>(a, 0, 1, ids[wave], share[wave]);
    __builtin_amdgcn_wave_barrier();
    if (blockIdx.x == 0 && n == 0 && wave == 0) {
        const int lane = threadIdx.x;
        const bool mine = lane < a.k && ids[0][lane] >= 0;
        if (lane < a.k) {
            a.ids[lane] = ids[0][lane];
            a.share[lane] = share[0][lane];
        }
        if (mine) {
            // experts come in the order of the slots, empty ones last
            a.active[lane] = ids[0][lane];
            a.begin[lane] = a.order[lane] = lane;
        }
        const int total = __popcll(__ballot(mine));
        if (lane == 0) {
            a.begin[total] = total;
            a.begin[a.most + 1] = total;
        }
    }
    const int e = uniform(ids[wave][n]);
    if (e < 0)
        return;
    up_tokens<MX, GATED, 1, 1>(
        a, e, blockIdx.x * (GATED ? 8 : 16), 1, [&](int) { return n; }, [&](int s) { return share[wave][s]; }, sums);
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

// Loads return in order, so a batch's weights (from memory) and h's values (from
// the L2) go out together, those of the next batch before this one's products.
// LDS: the sums of each wave and half, (waves, 2, tokens, 8), then active,
// begin and order.
// WHOLE: both halves of a sum over h are whole steps.  Else every load is checked,
// not the last step's alone, and the form spills (30 SGPRs and a VGPR, in MXFP8 47
// SGPRs): 5 tokens, 3 of 13 experts of 1111 x 333 12.2 us.
template <bool MX, bool WHOLE>
__global__ __launch_bounds__((MX ? kDownWavesMx : kDownWaves) * 64) void layer_down_kernel(LayerArgs a)
{
    typedef WeightStep<MX> Step;
    constexpr int WAVES = MX ? kDownWavesMx : kDownWaves, THREADS = WAVES * 64;
    constexpr int U = MX ? 2 : 3;  // what two batches' registers hold
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, fr = lane & 15, fk = lane >> 4, half = fr >> 3;
    float *sums = lds + wave * 2 * a.tokens * 8;
    int *active = reinterpret_cast<int *>(lds + WAVES * 2 * a.tokens * 8), *begin = active + a.most, *order = begin + a.most + 1;
    // all at once; entries past the last expert's are not looked at
    for (int i = threadIdx.x; i < a.tokens * a.k; i += THREADS)
        order[i] = a.order[i];
    for (int i = threadIdx.x; i <= a.most; i += THREADS) {
        if (i < a.most)
            active[i] = a.active[i];
        begin[i] = a.begin[i];
    }
    for (int i = lane; i < 2 * a.tokens * 8; i += 64)
        sums[i] = 0.0f;
    const int experts = uniform(a.begin[a.most + 1]);
    __syncthreads();
    // this lane's half of a sum over h
    const int d0 = blockIdx.x * 8, r = min(d0 + (fr & 7), a.width - 1);
    const int steps = (a.hidden + 2 * Step::K - 1) / (2 * Step::K), k0 = half * steps * Step::K;
    const char *rows = reinterpret_cast<const char *>(a.down.w) + r * a.down.sr * (MX ? 1 : 2);
    const uint8_t *scales = MX ? a.down.scales + r * a.down.ssr : nullptr;
    const int total = experts * steps, parts = a.splits * WAVES, own = blockIdx.y * WAVES + wave;
    const int end = uniform((int)((int64_t)total * (own + 1) / parts));

    // up to U steps of one expert, with h's values of its first 8 slots
    struct Batch {
        Step s[U];
        bf16x8 hi[U][Step::PIECES], lo[U][Step::PIECES];
        int n, j, steps;          // expert, first step, how many
        int first, count;         // its slots
    };
    // the slot in this lane's column of chunk c; past the last slot: that one
    // again, whose results are dropped
    auto slot_of = [&](const Batch &b, int c) { return order[b.first + min(c * 8 + (fr & 7), b.count - 1)]; };
    auto value = [&](const uint16_t *p, int k, int h) {
        return WHOLE ? token_piece<MX>(p, k, h) : token_piece_tail<MX>(p, k, h, a.hidden);
    };
    auto load = [&](Batch &b, int &i) {
        b.n = uniform(i / steps);
        b.j = i - b.n * steps;
        b.steps = min(min(steps - b.j, end - i), U);
        i += b.steps;
        const int64_t e = uniform(active[b.n]);
        b.first = uniform(begin[b.n]);
        b.count = uniform(begin[b.n + 1]) - b.first;
        const char *row = rows + e * a.down.se * (MX ? 1 : 2);
        const uint8_t *sc = MX ? scales + e * a.down.sse : nullptr;
        const int at = slot_of(b, 0) * a.hp;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + (b.j + min(u, b.steps - 1)) * Step::K;
            if (WHOLE)
                b.s[u].load(row, sc, k);
            else
                b.s[u].load_tail(row, sc, k, a.hidden);
#pragma unroll
            for (int h = 0; h < Step::PIECES; ++h) {
                b.hi[u][h] = value(a.hi + at, k, h);
                b.lo[u][h] = value(a.lo + at, k, h);
            }
        }
    };
    // to the tokens' sums; the two halves lie on the result's diagonal
    auto add = [&](const Batch &b, int c, float4v v) {
        if (c * 8 + (fr & 7) < b.count && (fk >> 1) == half) {
            const int t = slot_of(b, c) / a.k;
            float4v *to = reinterpret_cast<float4v *>(sums + (half * a.tokens + t) * 8 + (fk & 1) * 4);
            *to += v;
        }
    };
    const float4v zero = {0.0f, 0.0f, 0.0f, 0.0f};
    float4v acc = zero;
    // b's products; its expert's sums are done when the next batch is of another
    auto step = [&](const Batch &b, bool last) {
        auto products = [&](float4v sum, auto &&hi, auto &&lo) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < b.steps)
#pragma unroll
                    for (int h = 0; h < Step::PIECES; ++h) {
                        const bf16x8 w = b.s[u].piece(h);
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, lo(u, h), sum, 0, 0, 0);
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, hi(u, h), sum, 0, 0, 0);
                    }
            return sum;
        };
        acc = products(acc, [&](int u, int h) { return b.hi[u][h]; }, [&](int u, int h) { return b.lo[u][h]; });
        if (last) {
            add(b, 0, acc);
            acc = zero;
        }
        // more than 8 slots: chunk by chunk, straight to the tokens' sums
        for (int c = 1; c * 8 < b.count; ++c) {
            const int at = slot_of(b, c) * a.hp;
            add(b, c, products(zero, [&](int u, int h) { return value(a.hi + at, k0 + (b.j + u) * Step::K, h); },
                               [&](int u, int h) { return value(a.lo + at, k0 + (b.j + u) * Step::K, h); }));
        }
    };
    int i = uniform((int)((int64_t)total * own / parts));
    if (i < end) {
        Batch b0, b1;
        load(b0, i);
        for (;;) {
            if (i >= end) {
                step(b0, true);
                break;
            }
            load(b1, i);
            step(b0, b1.n != b0.n);
            if (i >= end) {
                step(b1, true);
                break;
            }
            load(b0, i);
            step(b1, b0.n != b1.n);
        }
    }
    __syncthreads();
    for (int at = threadIdx.x; at < a.tokens * 8; at += THREADS) {
        const int t = at >> 3, d = d0 + (at & 7);
        if (d >= a.width)
            continue;
        float v = 0.0f;
#pragma unroll 8
        for (int w = 0; w < 2 * WAVES; ++w)
            v += lds[w * a.tokens * 8 + at];
        if (a.splits > 1)
            a.parts[((int64_t)blockIdx.y * a.tokens + t) * a.width + d] = v;
        else
            layer_result(a, t, d, v);
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
