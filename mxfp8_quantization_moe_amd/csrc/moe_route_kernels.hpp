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
// The GPU times beside the kernels are medians of a kernel trace on one MI355X;
// an empty dependent kernel takes 2.3 us there and a large copy 4.9 TB/s.
//
// Three kernels.  The first gives each workgroup a run of tokens (at most
// kRouteMaxBlocks runs): L lanes hold a token's logits, V consecutive ones per
// lane, so the whole row stays in registers.  64 tokens at a time set their
// bits in one 64-bit mask per expert in LDS; a slot's rank among the run's
// slots of its expert is then a population count, whatever order the lanes ran
// in, and no atomic result depends on an order.  The second kernel scans the
// runs' counts and adds up their probabilities, the third adds the group
// starts to the ranks.  A single run (serving) does all of it in the first.
//
// The selection is bound by vector instructions, so it works on one unique
// key per logit: its order-preserving bits above the complement of its index.
// Equal logits then compare by index, and a key names its logit and expert: a
// bf16 logit's key has 32 bits, an fp32 logit's is the bit pattern of a
// positive double (numerical order = order of the bits), and minima and maxima
// need no comparison flags.  Each lane sorts its V keys once in a network;
// every slot takes the largest head over the token's lanes and moves the
// winner's list up.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_rows_kernels.hpp"
#include "mxq_device.hpp"
#include "wave_ops.hpp"

namespace mxq {

constexpr int kRouteTile = 64;        // tokens that share one round of bit masks
constexpr int kRouteMaxBlocks = 256;  // runs of tokens (workgroups of the first kernel)
constexpr int kNoExpert = 0xffff;
constexpr float kLog2E = 1.4426950408889634f;
constexpr int kScanThreads = 1024;    // workgroups of the second kernel: 16 experts x 64 parts of the runs
constexpr int kScanExperts = 16;
constexpr int kPlaceThreads = 256;    // workgroups of the third kernel

// order-preserving bits of fp32 (-0 equals +0: adding zero makes it +0)
__device__ __forceinline__ uint32_t ordered_bits(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t b)
{
    return __uint_as_float(b ^ (b >> 31 ? 0x80000000u : 0xffffffffu));
}

// Unique keys of the logits of type T, NaN as -inf.  Keys below kFirst are -inf's.
template <typename T>
struct RouteKey;
template <>
struct RouteKey<uint16_t> {
    typedef uint32_t K;
    static constexpr K kFirst = 0x00800000u;  // -inf: 0x007f....
    static __device__ __forceinline__ K make(float v, int e)
    {
        return (ordered_bits(fmaxf(v, -INFINITY)) & 0xffff0000u) | (uint32_t)(0xffff - e);
    }
    static __device__ __forceinline__ K big(K a, K b) { return a > b ? a : b; }
    static __device__ __forceinline__ K small(K a, K b) { return a < b ? a : b; }
    static __device__ __forceinline__ int expert(K k) { return 0xffff - (int)(k & 0xffffu); }
    // the low half of a negative value's order-preserving bits was ones
    static __device__ __forceinline__ float logit(K k)
    {
        return from_ordered(k >> 31 ? k & 0xffff0000u : k | 0xffffu);
    }
    template <int CTRL>
    static __device__ __forceinline__ K move(K k) { return dpp<CTRL>(k); }
    static __device__ __forceinline__ K xor_lane(K k, int m) { return (K)__shfl_xor((int)k, m, 64); }
};
template <>
struct RouteKey<float> {
    typedef double K;
    // bits 61..30: the logit's, 29..18: the index's (below 4096); the top two
    // bits are 0, so every key is a positive finite double
    static constexpr K kFirst = 0x1p-1021;    // bits of 0x00800000 << 30 (-inf: 0x007fffff << 30)
    static __device__ __forceinline__ K make(float v, int e)
    {
        const uint64_t b =
            (uint64_t)ordered_bits(fmaxf(v, -INFINITY)) << 30 | (uint64_t)(uint32_t)(4095 - e) << 18;
        return __longlong_as_double((long long)b);
    }
    static __device__ __forceinline__ K big(K a, K b) { return __builtin_fmax(a, b); }
    static __device__ __forceinline__ K small(K a, K b) { return __builtin_fmin(a, b); }
    static __device__ __forceinline__ int expert(K k)
    {
        return 4095 - (int)((uint64_t)__double_as_longlong(k) >> 18 & 4095u);
    }
    static __device__ __forceinline__ float logit(K k)
    {
        return from_ordered((uint32_t)((uint64_t)__double_as_longlong(k) >> 30));
    }
    template <int CTRL>
    static __device__ __forceinline__ K move(K k)
    {
        const uint64_t b = (uint64_t)__double_as_longlong(k);
        return __longlong_as_double((long long)((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b)));
    }
    static __device__ __forceinline__ K xor_lane(K k, int m) { return __shfl_xor(k, m, 64); }
};

// reductions over aligned groups of L lanes; every lane gets the result
template <int L, typename F, typename M, typename X>
__device__ __forceinline__ F lanes_reduce(F v, M &&op, X &&xor_lane)
{
    if constexpr (L >= 2) v = op(v, std::integral_constant<int, kDppQuadXor1>());
    if constexpr (L >= 4) v = op(v, std::integral_constant<int, kDppQuadXor2>());
    if constexpr (L >= 8) v = op(v, std::integral_constant<int, kDppHalfMirror>());
    if constexpr (L >= 16) v = op(v, std::integral_constant<int, kDppRowMirror>());
    if constexpr (L >= 32) v = xor_lane(v, 16);
    if constexpr (L >= 64) v = xor_lane(v, 32);
    return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    return lanes_reduce<L>(
        v, [](float x, auto c) { return x + __uint_as_float(dpp<c()>(__float_as_uint(x))); },
        [](float x, int m) { return x + __shfl_xor(x, m, 64); });
}

template <int L>
__device__ __forceinline__ float lanes_max(float v)
{
    return lanes_reduce<L>(
        v, [](float x, auto c) { return fmaxf(x, __uint_as_float(dpp<c()>(__float_as_uint(x)))); },
        [](float x, int m) { return fmaxf(x, __shfl_xor(x, m, 64)); });
}

template <int L, typename T>
__device__ __forceinline__ typename RouteKey<T>::K lanes_best(typename RouteKey<T>::K v)
{
    typedef RouteKey<T> R;
    return lanes_reduce<L>(
        v, [](typename R::K x, auto c) { return R::big(x, R::template move<c()>(x)); },
        [](typename R::K x, int m) { return R::big(x, R::xor_lane(x, m)); });
}

// Batcher's odd-even merge sort of the first N keys (a power of two), largest
// first
template <typename T, int N, int M>
__device__ __forceinline__ void sort_keys(typename RouteKey<T>::K (&k)[M])
{
    typedef RouteKey<T> R;
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const typename R::K a = k[i + j], b = k[i + j + q];
                        k[i + j] = R::big(a, b);
                        k[i + j + q] = R::small(a, b);
                    }
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

// Workspace of a call.  Per run, the counts of every expert (after the second
// kernel: those of the runs before), their probability sums, the sum of lse^2
// and the number of live tokens; per expert its share of the balance loss.
struct RouteWorkspace {
    int32_t *counts;  // [runs][experts]
    float *probs;     // [runs][experts]
    float *z;         // [runs]
    int32_t *live;    // [runs]
    double *balance;  // [experts]
};

struct RouteResults {
    int32_t *counts, *offs;
    float *mean_prob, *losses;
    int32_t *live;
};

// Group ends and starts from the counts (start may be count), by one wave:
// consecutive experts per lane, one scan of the lanes' sums.
__device__ __forceinline__ void group_ends(const int32_t *count, int32_t *start, int32_t *offs, int experts, int align)
{
    const int lane = threadIdx.x & 63, per = (experts + 63) / 64;
    const int e0 = min(lane * per, experts), e1 = min(e0 + per, experts);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        sum += (count[e] + align - 1) / align * align;
    int upto = sum;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int up = __shfl_up(upto, m, 64);
        upto += lane >= m ? up : 0;
    }
    int at = upto - sum;
    for (int e = e0; e < e1; ++e) {
        const int next = at + (count[e] + align - 1) / align * align;
        start[e] = at;
        if (offs)
            offs[e] = next;
        at = next;
    }
}

// One run of tokens per workgroup.  L lanes per token, V experts per lane.
// FEW: at most 8 slots, so only the first 8 of a lane's sorted keys can be
// taken.  ONE: the only run.
// 16384 tokens x 256 experts fp32, 8 slots: 19 us for 19 MB.  Vector
// instructions (1060 per wave of 4 tokens; 640 with bf16 logits' 32-bit keys)
// issue in 44% of the cycles; the waves wait in 61% of theirs: one workgroup
// per CU has one round, whose load, reductions, selection, ranks and closing
// sum follow one another.  x 8 experts bf16, 2 slots: 4.4 us, latency; one
// token of 256: 7.6 us, its chain of reductions.
template <typename T, int L, int V, bool FEW, int THREADS, bool ONE>
__global__ __launch_bounds__(THREADS) void moe_route_kernel(
    const T *__restrict__ logits, int64_t sl, int tokens, int experts, const uint8_t *__restrict__ mask, int k,
    int renorm, int align, int run, int32_t *__restrict__ ids, float *__restrict__ weights,
    int32_t *__restrict__ rows, float *__restrict__ lse_out, RouteWorkspace ws, RouteResults out)
{
    typedef RouteKey<T> R;
    typedef typename R::K K;
    constexpr int G = THREADS / L;  // tokens in flight
    constexpr int WAVES = THREADS / 64;
    // slots a lane keeps: slot j stays with lane j % L of its token
    constexpr int KEEP = FEW || L >= 32 ? 1 : 32 / L, D = FEW && V > 8 ? 8 : V;
    // per expert the 64-token mask and the run's count so far; per slot of the
    // round its weight and expert
    extern __shared__ uint64_t lds[];
    uint64_t *bits = lds;
    int32_t *count = reinterpret_cast<int32_t *>(bits + experts);
    float *slot_w = reinterpret_cast<float *>(count + experts);
    uint16_t *slot_e = reinterpret_cast<uint16_t *>(slot_w + kRouteTile * k);
    __shared__ float zpart[WAVES], npart[WAVES];
    const int tid = threadIdx.x, sub = tid % L, wave = tid >> 6, lane = tid & 63;
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
    // the end of a whole last run, and the step past its last round, may not
    // fit 31 bits: rounds are counted by the tokens left
    const int first = blockIdx.x * run, own = min(run, tokens - first);
    for (int t0 = first, left = own; ONE ? t0 == first : left > 0;
         t0 = (int)((uint32_t)t0 + kRouteTile), left -= kRouteTile) {
        // s0: the wave's first token, so that the wave leaves together
        for (int s0 = wave * (64 / L); s0 < min(kRouteTile, left); s0 += G) {
            const int s = s0 + lane / L, t = t0 + s;
            const bool in = s < left;
            const int tl = in ? t : first;
            float v[V];
            load_row<T, V>(logits + (int64_t)tl * sl, e0, experts, whole, -INFINITY, v);
            bool live = in && (!mask || mask[tl] != 0);
            float top = v[0];
#pragma unroll
            for (int i = 1; i < V; ++i)
                top = fmaxf(top, v[i]);
            top = lanes_max<L>(top);
            // fmax drops NaN: a row of -inf and NaN alone has no logit either
            live = live && top > -INFINITY;
            // exp(v - top), the difference first: that of two finite logits
            // overflows to -inf alone, which is right, while top log2 e
            // overflows for |top| past 2.36e38 (rows barred with the type's
            // lowest value)
            float p[V], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = __builtin_amdgcn_exp2f((v[i] - top) * kLog2E);
                sum += p[i];
            }
            sum = lanes_sum<L>(sum);
            const float lse = live ? logf(sum) + top : INFINITY;
            const float inv = live ? 1.0f / sum : 0.0f;
            if (live) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] = fmaf(p[i], inv, acc[i]);
                if (sub == 0) {
                    zsum = fmaf(lse, lse, zsum);
                    ++nlive;
                }
            }
            if (sub == 0 && in)
                lse_out[t] = lse;
            // and a 0 after the last: moving a list up then has one form for every
            // entry.  As a choice of the index it was compiled into a search of
            // all entries per move (262144 x 128 bf16, 8 slots: 148 us, now 89)
            K key[V + 1];
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = R::make(v[i], e0 + i);
            key[V] = (K)0;
            if constexpr (V <= 16)
                sort_keys<T, V>(key);
            K kept[KEEP];
#pragma unroll
            for (int q = 0; q < KEEP; ++q)
                kept[q] = (K)0;
#pragma unroll
            for (int q = 0; q < KEEP; ++q)
                for (int j = q * L; j < min(k, (q + 1) * L); ++j) {
                    K best = key[0];
                    if constexpr (V > 16) {
#pragma unroll
                        for (int i = 1; i < V; ++i)
                            best = R::big(best, key[i]);
                    }
                    const K win = lanes_best<L, T>(best);
                    if constexpr (V > 16) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            key[i] = key[i] == win ? (K)0 : key[i];
                    } else {
                        const bool mine = key[0] == win;
#pragma unroll
                        for (int i = 0; i < D; ++i)
                            key[i] = mine ? key[i + 1] : key[i];
                    }
                    kept[q] = sub + q * L == j ? win : kept[q];
                }
            float w[KEEP], total = 0.0f;
#pragma unroll
            for (int q = 0; q < KEEP; ++q) {
                const bool taken = live && kept[q] >= R::kFirst;
                w[q] = taken ? __builtin_amdgcn_exp2f((R::logit(kept[q]) - top) * kLog2E) * inv : 0.0f;
                total += w[q];
            }
            const float norm = renorm ? 1.0f / lanes_sum<L>(total) : 1.0f;
#pragma unroll
            for (int q = 0; q < KEEP; ++q) {
                const int j = sub + q * L;
                if (j < k) {
                    const bool taken = live && kept[q] >= R::kFirst;
                    const int e = R::expert(kept[q]);
                    slot_w[s * k + j] = taken ? w[q] * norm : 0.0f;
                    slot_e[s * k + j] = taken ? (uint16_t)e : (uint16_t)kNoExpert;
                    if (taken)
                        atomicOr(reinterpret_cast<unsigned long long *>(bits + e), 1ull << s);
                }
            }
        }
        __syncthreads();
        if constexpr (ONE) {
            for (int e = tid; e < experts; e += THREADS) {
                const int c = __popcll(bits[e]);
                count[e] = c;
                out.counts[e] = c;
            }
            __syncthreads();
            if (tid < 64)
                group_ends(count, count, out.offs, experts, align);
            __syncthreads();
        }
        // rank of each slot among the run's slots of its expert
        const int n = min(kRouteTile, left) * k;
        for (int i = tid; i < n; i += THREADS) {
            const int s = i / k;
            const int64_t at = (int64_t)t0 * k + i;
            const int e = slot_e[i];
            const bool taken = e != kNoExpert;
            ids[at] = taken ? e : -1;
            weights[at] = slot_w[i];
            rows[at] = taken ? count[e] + __popcll(bits[e] & ((1ull << s) - 1)) : -1;
        }
        __syncthreads();
        if constexpr (!ONE) {
            for (int e = tid; e < experts; e += THREADS) {
                count[e] += __popcll(bits[e]);
                bits[e] = 0;
            }
            __syncthreads();
        }
    }
    // the run's sums: lanes that hold the same experts, then the waves two by
    // two, so that their order is fixed
    float *psum = reinterpret_cast<float *>(bits);  // two sets
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int m = L; m < 64; m <<= 1)
            acc[i] += __shfl_xor(acc[i], m, 64);
    zsum = lanes_sum<64>(zsum);
    const float fl = lanes_sum<64>((float)nlive);
    if (lane == 0) {
        zpart[wave] = zsum;
        npart[wave] = fl;
    }
    const int waves = min(WAVES, (min(own, kRouteTile) + 64 / L - 1) / (64 / L));  // that had a token
    for (int w = 0; w < max(waves, 2); w += 2) {
        if (wave >> 1 == w >> 1 && lane < L) {
            float *set = psum + (wave & 1) * experts;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < experts)
                    set[e0 + i] = (w ? set[e0 + i] : 0.0f) + acc[i];
        }
        __syncthreads();
    }
    float z = 0.0f, nl = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        z += zpart[w];
        nl += npart[w];
    }
    if constexpr (!ONE) {
        for (int e = tid; e < experts; e += THREADS) {
            ws.counts[(int64_t)blockIdx.x * experts + e] = count[e];
            ws.probs[(int64_t)blockIdx.x * experts + e] = psum[e] + psum[experts + e];
        }
        if (tid == 0) {
            ws.z[blockIdx.x] = z;
            ws.live[blockIdx.x] = (int)nl;
        }
    } else {
        const double inv = nl > 0.0f ? 1.0 / (double)nl : 0.0;
        double b = 0.0;
        for (int e = tid; e < experts; e += THREADS) {
            const double p = (double)(psum[e] + psum[experts + e]) * inv;
            out.mean_prob[e] = (float)p;
            b += (double)out.counts[e] * p;  // this thread's own store
        }
        __shared__ double part[WAVES];
        b = block_sum<THREADS>(part, b);
        if (tid == 0) {
            out.losses[0] = (float)(b * (double)experts * inv / (double)k);
            out.losses[1] = (float)((double)z * inv);
            out.live[0] = (int)nl;
        }
    }
}

// 16 experts per workgroup, 64 threads each, every thread a contiguous part of
// the runs: counts of the runs before each run (in place), totals, mean
// probabilities (64-bit sums in a fixed order).  Bound by its chain of
// latencies, so all of a thread's loads are issued first: 5.1 us for 256 runs
// of 256 experts; with 32 experts per workgroup 1 us more.
__global__ __launch_bounds__(kScanThreads) void moe_scan_kernel(int experts, int nruns, RouteWorkspace ws,
                                                                RouteResults out)
{
    constexpr int PARTS = kScanThreads / kScanExperts, MOST = kRouteMaxBlocks / PARTS;
    __shared__ int32_t psum[PARTS][kScanExperts + 1];
    __shared__ double qsum[PARTS][kScanExperts + 1];
    __shared__ int32_t alive[kScanThreads / 64];
    const int tid = threadIdx.x, part = tid / kScanExperts, x = tid % kScanExperts;
    const int e = blockIdx.x * kScanExperts + x;
    const int per = (nruns + PARTS - 1) / PARTS, r0 = min(part * per, nruns), r1 = min(r0 + per, nruns);
    int c[MOST], sum = 0;
    float q[MOST];
    double p = 0.0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const bool on = r0 + i < r1 && e < experts;
        const int64_t at = (int64_t)(r0 + i) * experts + e;
        c[i] = on ? ws.counts[at] : 0;
        q[i] = on ? ws.probs[at] : 0.0f;
    }
    int own = tid < nruns ? ws.live[tid] : 0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        own += __shfl_xor(own, m, 64);
    if (tid % 64 == 0)
        alive[tid / 64] = own;
#pragma unroll
    for (int i = 0; i < MOST; ++i)
        p += (double)q[i];
#pragma unroll
    for (int i = 0; i < MOST; ++i)
        sum += c[i];
    psum[part][x] = sum;
    qsum[part][x] = p;
    __syncthreads();
    {
        // the parts of one expert in consecutive lanes: one scan
        const int q = tid % PARTS, y = tid / PARTS;
        const int own = psum[q][y];
        double all = qsum[q][y];
        int upto = own;
#pragma unroll
        for (int m = 1; m < PARTS; m <<= 1) {
            const int up = __shfl_up(upto, m, PARTS);
            upto += q >= m ? up : 0;
            all += __shfl_xor(all, m, PARTS);
        }
        psum[q][y] = upto - own;
        const int f = blockIdx.x * kScanExperts + y;
        if (q == PARTS - 1 && f < experts) {
            int n = 0;
            for (int w = 0; w < (nruns + 63) / 64; ++w)
                n += alive[w];
            const double inv = n > 0 ? 1.0 / (double)n : 0.0;
            out.counts[f] = upto;
            out.mean_prob[f] = (float)(all * inv);
            ws.balance[f] = (double)upto * (all * inv);
        }
    }
    __syncthreads();
    int before = psum[part][x];
#pragma unroll
    for (int i = 0; i < MOST; ++i)
        if (r0 + i < r1 && e < experts) {
            ws.counts[(int64_t)(r0 + i) * experts + e] = before;
            before += c[i];
        }
}

// A run per workgroup: its slots' ranks become rows.  The last workgroup
// writes the group ends and the losses.  4.2 us for 131072 slots of 256
// experts, latency (1.8 MB).
__global__ __launch_bounds__(kPlaceThreads) void moe_place_kernel(int tokens, int experts, int k, int align, int run,
                                                                  int nruns, const int32_t *__restrict__ ids,
                                                                  int32_t *__restrict__ rows, RouteWorkspace ws,
                                                                  RouteResults out)
{
    extern __shared__ uint64_t lds[];
    int32_t *start = reinterpret_cast<int32_t *>(lds);  // [experts]
    const int tid = threadIdx.x, r = blockIdx.x;
    const bool final = r == nruns;
    for (int e = tid; e < experts; e += kPlaceThreads)
        start[e] = out.counts[e];
    __syncthreads();
    if (tid < 64)
        group_ends(start, start, final ? out.offs : nullptr, experts, align);
    __syncthreads();
    if (final) {
        __shared__ double part[kPlaceThreads / 64];
        double z = 0.0, b = 0.0, n = 0.0;
        for (int i = tid; i < nruns; i += kPlaceThreads) {
            z += (double)ws.z[i];
            n += (double)ws.live[i];
        }
        for (int e = tid; e < experts; e += kPlaceThreads)
            b += ws.balance[e];
        z = block_sum<kPlaceThreads>(part, z);
        n = block_sum<kPlaceThreads>(part, n);
        b = block_sum<kPlaceThreads>(part, b);
        if (tid == 0) {
            const double inv = n > 0.0 ? 1.0 / n : 0.0;
            out.losses[0] = (float)(b * (double)experts * inv / (double)k);
            out.losses[1] = (float)(z * inv);
            out.live[0] = (int)n;
        }
        return;
    }
    const int64_t first = (int64_t)r * run * k, last = min((int64_t)(r + 1) * run, (int64_t)tokens) * k;
    for (int64_t i = first + tid; i < last; i += kPlaceThreads) {
        const int e = ids[i];
        if (e >= 0)
            rows[i] += start[e] + ws.counts[(int64_t)r * experts + e];
    }
}

// The second and third kernel in one, for few runs and experts: every
// workgroup adds up all the runs' counts itself, each expert by several
// threads (integer sums, in any order).  6.2 us for 256 runs of 8 experts,
// 8.4 for 65 of 61: latency, against two launches saved into one.
__global__ __launch_bounds__(kPlaceThreads) void moe_finish_kernel(int tokens, int experts, int k, int align, int run,
                                                                   int nruns, const int32_t *__restrict__ ids,
                                                                   int32_t *__restrict__ rows, RouteWorkspace ws,
                                                                   RouteResults out)
{
    extern __shared__ uint64_t lds[];
    const int tid = threadIdx.x, r = blockIdx.x;
    const bool final = r == nruns;
    const int parts = max(1, kPlaceThreads / experts);
    double *qsum = reinterpret_cast<double *>(lds);                      // [parts][experts]
    int32_t *total = reinterpret_cast<int32_t *>(qsum + parts * experts);  // [experts] counts, then starts
    int32_t *before = total + experts;                                   // [experts] in earlier runs
    for (int e = tid; e < 2 * experts; e += kPlaceThreads)
        total[e] = 0;
    __syncthreads();
    for (int i = tid; i < parts * experts; i += kPlaceThreads) {
        const int e = i % experts, part = i / experts;
        int all = 0, prior = 0;
        double p = 0.0;
#pragma unroll 8
        for (int q = part; q < nruns; q += parts) {
            const int64_t at = (int64_t)q * experts + e;
            const int c = ws.counts[at];
            all += c;
            prior += q < r ? c : 0;
            if (final)
                p += (double)ws.probs[at];
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], prior);
        if (final)
            qsum[i] = p;
    }
    __syncthreads();
    if (final) {
        __shared__ double part[kPlaceThreads / 64];
        double z = 0.0, n = 0.0, b = 0.0;
        for (int i = tid; i < nruns; i += kPlaceThreads) {
            z += (double)ws.z[i];
            n += (double)ws.live[i];
        }
        z = block_sum<kPlaceThreads>(part, z);
        n = block_sum<kPlaceThreads>(part, n);
        const double inv = n > 0.0 ? 1.0 / n : 0.0;
        for (int e = tid; e < experts; e += kPlaceThreads) {
            double p = 0.0;
            for (int i = 0; i < parts; ++i)
                p += qsum[i * experts + e];
            p *= inv;
            out.counts[e] = total[e];
            out.mean_prob[e] = (float)p;
            b += (double)total[e] * p;
        }
        b = block_sum<kPlaceThreads>(part, b);
        if (tid == 0) {
            out.losses[0] = (float)(b * (double)experts * inv / (double)k);
            out.losses[1] = (float)(z * inv);
            out.live[0] = (int)n;
        }
    }
    if (tid < 64)
        group_ends(total, total, final ? out.offs : nullptr, experts, align);
    __syncthreads();
    if (final)
        return;
    const int64_t first = (int64_t)r * run * k, last = min((int64_t)(r + 1) * run, (int64_t)tokens) * k;
    for (int64_t i = first + tid; i < last; i += kPlaceThreads) {
        const int e = ids[i];
        if (e >= 0)
            rows[i] += total[e] + before[e];
    }
}

// |lse| up to which its rounding to fp32 matters no more than that of an
// exponential (see moe_route_backward_kernel)
constexpr float kNearLse = 16.0f;

// words from one lane's entries to the next lane's in a row of LDS
constexpr int route_row_step(int v) { return v > 4 && v <= 16 ? v + 4 : v; }

// dl_te = p_te (g_te - sum_e' p_te' g_te') + 2 g_z lse_t p_te / n with
// g_te = g_b E c_e / (n^2 k) + [e = ids_tj] q_tj, where q is the gradient of
// the selected probabilities (through the renormalisation when there is one).
// A slot's part is worked out by one lane and reaches the lane that holds its
// expert through a row of zeros in LDS (comparing every expert with every slot
// took three times as long).  16384 x 256 fp32: 13.6 us for 35 MB (2.6 TB/s);
// 65536 x 256 bf16 21.6 us (3.2 TB/s): one pass over the memory, each group of
// lanes with one token at a time, bound by the latency of its chain (vector
// instructions issue in 28% of the first one's cycles, its waves wait in 63%).
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(
    const T *__restrict__ logits, int64_t sl, int tokens, int experts, int k, int renorm,
    const int32_t *__restrict__ ids, const float *__restrict__ weights, const float *__restrict__ lse_in,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ live, const float *__restrict__ gw,
    const float *__restrict__ gl, T *__restrict__ dl, int64_t sd)
{
    extern __shared__ uint64_t lds[];
    const int tid = threadIdx.x, sub = tid % L, e0 = sub * V;
    const bool whole = experts % V == 0;
    // this token's row, V entries per lane; 4 words between lanes' entries
    // spread the 16-byte reads of 16 lanes over all banks
    constexpr int STEP = route_row_step(V);
    float *row = reinterpret_cast<float *>(lds) + tid / L * (L * STEP), *mine = row + sub * STEP;
    auto entry = [&](int e) -> float & { return row[e / V * STEP + e % V]; };
#pragma unroll
    for (int i = 0; i < V; ++i)
        mine[i] = 0.0f;
    const float n = (float)max(live ? live[0] : 1, 1);
    const float gb = gl ? gl[0] * (float)experts / (n * (float)k) / n : 0.0f;
    const float gz = gl ? 2.0f * gl[1] / n : 0.0f;
    float bal[V];
    if (gl && whole && e0 < experts) {
        typedef int32_t Ints __attribute__((ext_vector_type(V), aligned(4)));
        const Ints c = *reinterpret_cast<const Ints *>(counts + e0);
#pragma unroll
        for (int i = 0; i < V; ++i)
            bal[i] = gb * (float)c[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            bal[i] = gl && e0 + i < experts ? gb * (float)counts[e0 + i] : 0.0f;
    }
    const int64_t per_grid = (int64_t)gridDim.x * (256 / L);
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + tid / L; t < tokens; t += per_grid) {
        float v[V];
        load_row<T, V>(logits + t * sl, e0, experts, whole, -INFINITY, v);
        const float lse = lse_in[t];
        const bool dead = lse == INFINITY;
        if (gw) {
            float total = 0.0f, wg = 0.0f;
            if (renorm) {
                for (int j = sub; j < k; j += L) {
                    const int e = ids[t * k + j];
                    if (e >= 0 && e < experts) {
                        total += __expf(Piece<T>::to_f32(logits[t * sl + e]) - lse);
                        wg = fmaf(weights[t * k + j], gw[t * k + j], wg);
                    }
                }
                total = lanes_sum<L>(total);
                wg = lanes_sum<L>(wg);
            }
            const float inv = renorm ? 1.0f / total : 1.0f;
            for (int j = sub; j < k; j += L) {
                const int e = ids[t * k + j];
                if (e >= 0 && e < experts)
                    entry(e) = (gw[t * k + j] - wg) * inv;
            }
            // lanes of one wave: LDS runs its instructions in order
            __builtin_amdgcn_wave_barrier();
        }
        float p[V], g[V], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            p[i] = __expf(v[i] - lse);  // 0 for -inf; a dead token's is not used
        // lse is rounded to fp32: these p are off by half its last place,
        // 2^-21 at most up to kNearLse.  From there on their sum takes that
        // factor out again (it stays below 4096 however large lse is: rounding
        // moves lse no further than the largest logit), and out of the q that
        // were divided by such a sum.  For every token it would cost 262144 x
        // 64 bf16 29.4 us, 28.1 so (27.0 without); 16384 x 256 fp32 14.1, 13.6.
        if (!dead && fabsf(lse) > kNearLse) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum += p[i];
            sum = lanes_sum<L>(sum);
            const float scale = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] *= scale;
                if (gw && renorm)
                    mine[i] *= sum;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = bal[i] + (gw ? mine[i] : 0.0f);
            dot = fmaf(p[i], g[i], dot);
        }
        dot = lanes_sum<L>(dot);
        if (gw) {
            __builtin_amdgcn_wave_barrier();
            for (int j = sub; j < k; j += L) {
                const int e = ids[t * k + j];
                if (e >= 0 && e < experts)
                    entry(e) = 0.0f;
            }
            __builtin_amdgcn_wave_barrier();
        }
        typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
        T *out = dl + t * sd + e0;
        Vec o;
#pragma unroll
        for (int i = 0; i < V; ++i)
            // (2 g_z p) lse: 0 for p = 0 whatever 2 g_z lse comes to
            o[i] = Piece<T>::from_f32(dead ? 0.0f : fmaf(gz * p[i], lse, p[i] * (g[i] - dot)));
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
