// Routing of tokens to experts: scores, the k best experts of every token with
// their weights, the rows sorted by expert with the experts' offsets, and the
// gradient of the logits.
//
// Up to 8 choices of up to 512 experts (route_kernel): 8, 16 or 32 lanes a token,
// each with up to 16 neighbouring experts of one group.  A value becomes a 32-bit
// key, its order-preserving bits above the expert's index, so that every key is
// different and a comparison is one instruction; a lane sorts its keys by a
// network, keeps eight, and the lanes merge their lists in 3 to 5 exchanges.  BF16
// logits fit their key whole; of FP32 values it holds 23 bits, and the chosen are
// put in order by their full values afterwards.  (One pick after another by
// warp-wide maxima took 780 instructions a token of 128 experts and 2300 of 256 in
// groups; 194 and 847 now.)  Neither memory (8 to 10 % of its rate) nor the issue of
// instructions (47 to 52 %) is used up: with the 32 warps an SM that 64 registers
// leave, the latency of loads and exchanges and the slowest warp before a CTA's
// barrier set the time: 16384 tokens of 256 experts 23 us, 32768 of 128 11 us, both
// without the sorting by expert (6 us).
// What the keys, or FP32 itself, leave open (a key equal in its 23 bits to the last
// choice's, or a sum with a bias nearer than a bound on the rounding of the scores:
// one token in a hundred) is settled by settle_token: the few experts that may be
// among the chosen, one a lane, are ranked by their values, in FP64 where FP32
// cannot tell two apart.  Sums of groups that are as near are taken again in FP64;
// softmax scores that near, more choices and more experts take route_slowly, a warp
// a token: 16384 tokens with 9 choices of 128 experts 39 us (8 choices 15), with 10
// of 512 45 us, with 8 of 256 by softmax and a bias 58 us (by sigmoid 28).  The
// bound on the rounding goes by the largest finite bias: with one of -1e9 every
// sum is near another, and those tokens take 0.4 to 1.1 ms (minus infinity: 30 us).
//
// Sorting by expert is a counting sort, stable and without atomics whose order
// would matter: CTA c routes a run of tokens and counts its choices by expert;
// a second launch adds the counts of the CTAs before it, and places its own
// run, warp by warp, with a warp-wide match for the rank among 32 choices.
// Where one CTA does all tokens, both steps are one launch.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "../../include/gemm_route.h"
#include "launch.h"
#include "ptx.cuh"
#include "route.h"

namespace dg {
namespace {

constexpr float kTiny = 1e-20f;  // added to the sum of chosen sigmoid scores
constexpr unsigned kFull = 0xffffffffu;

struct RouteParams {
    const void *logits;
    long long ld;
    int tokens, experts, k;
    const float *bias;
    int groups, top_groups, per_group;
    int sigmoid, renormalise;
    float scale;
    float *weights;
    long long *expert, *order, *offsets;
    int *counts;
    int chunks, per_chunk;  // CTAs, tokens of each
    int pitch;              // of a CTA's row of counts
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Integers in the order of the values; 0 stands for "no choice", below minus
// infinity's neighbours.  Negative zero counts as zero.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x == -INFINITY ? 0u : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k == 0u ? -INFINITY : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x)
{
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return x == -INFINITY ? 0u : u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k)
{
    const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, d));
    return x;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    return x;
}

// The two largest of all lanes' two.
template <typename F>
__device__ __forceinline__ void warp_top2(F &a, F &b)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const F a2 = __shfl_xor_sync(kFull, a, d), b2 = __shfl_xor_sync(kFull, b, d);
        const F low = a < a2 ? a : a2, best = b < b2 ? b2 : b;
        b = low < best ? best : low;
        a = a < a2 ? a2 : a;
    }
}

// The n first of the keys (expert j * 32 + lane in key[j], 0 none), equal ones
// by index: lane i gets pick i's key and index (-1: none).
template <int V, typename Key>
__device__ __forceinline__ void pick(Key (&key)[V], int n, int lane, Key &my_key, int &my_index)
{
    my_key = 0;
    my_index = -1;
    Key top = 0;
    int at = 0;
    const auto rescan = [&]() {
        top = key[0];
        at = 0;
#pragma unroll
        for (int j = 1; j < V; ++j)
            if (key[j] > top) {
                top = key[j];
                at = j;
            }
    };
    rescan();
    for (int i = 0; i < n; ++i) {
        const Key best = warp_max_key(top);
        if (best == 0) break;
        const uint32_t index = __reduce_min_sync(kFull, top == best ? static_cast<uint32_t>(at * 32 + lane) : kFull);
        if (lane == i) {
            my_key = best;
            my_index = static_cast<int>(index);
        }
        if ((index & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == static_cast<int>(index >> 5)) key[j] = 0;
            rescan();
        }
    }
}

// The choice of a row in FP64: lane i < k gets pick i.
template <int V, typename T>
__device__ __noinline__ int choose_exactly(const RouteParams &p, const T *row, int lane)
{
    double v[V];
    float top = -INFINITY;
    for (int j = 0; j < V; ++j) {
        const int e = j * 32 + lane;
        const float x = e < p.experts ? to_float(row[e]) : -INFINITY;
        v[j] = x;
        top = fmaxf(top, x);
    }
    top = warp_max(top);
    double sum = 0.0;
    if (!p.sigmoid) {
        for (int j = 0; j < V; ++j)
            if (v[j] != -INFINITY) sum += exp(v[j] - top);
        sum = warp_sum(sum);
    }
    uint64_t key[V];
    for (int j = 0; j < V; ++j) {
        const int e = j * 32 + lane;
        const double b = p.bias && e < p.experts ? static_cast<double>(p.bias[e]) : 0.0;
        if (v[j] != -INFINITY) v[j] = (p.sigmoid ? 1.0 / (1.0 + exp(-v[j])) : exp(v[j] - top) / sum) + b;
        key[j] = key_of(v[j]);
    }
    if (p.groups > 1) {
        double score = -INFINITY;  // of group `lane`
        for (int g = 0; g < p.groups; ++g) {
            double a = -INFINITY, b = -INFINITY;
            for (int j = 0; j < V; ++j)
                if ((j * 32 + lane) / p.per_group == g) {
                    b = fmax(b, fmin(a, v[j]));
                    a = fmax(a, v[j]);
                }
            warp_top2(a, b);
            if (lane == g) score = b == -INFINITY ? a : a + b;
        }
        uint64_t gkey[1] = {key_of(score)}, unused;
        int open;
        pick<1>(gkey, p.top_groups, lane, unused, open);
        const uint32_t kept = __reduce_or_sync(kFull, open >= 0 ? 1u << open : 0u);
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            if (e < p.experts && !((kept >> (e / p.per_group)) & 1u)) key[j] = 0;
            // without a bias the ranking is the logits' own
            if (!p.bias && key[j]) key[j] = key_of(static_cast<double>(to_float(row[e])));
        }
    }
    uint64_t unused;
    int index;
    pick<V>(key, p.k, lane, unused, index);
    return index;
}

// For the ranking alone: e^x to 2^-22 and x * 2^-24, 1 / x to an ulp, flushed.
__device__ __forceinline__ float exp_near(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950409f));
    return y;
}
__device__ __forceinline__ float inverse_near(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How far two scores plus biases may be off, together, from what they stand for:
// FP32 exp (2 ulp), addition and division of a sigmoid and the bias's addition; for
// a softmax also the sum of up to V / 32 + 5 roundings and the exponent's.  Below
// 2^-125 a fast division gives zero: 2^-126 for each of a group's two best.
__device__ __forceinline__ float score_bound(const RouteParams &p, float most, float bias_max)
{
    return (most + bias_max) * (p.sigmoid ? 1e-6f : 4e-6f) + 4e-38f;
}

// A group's score from its two best (minus infinity: none).  Biases of the type's
// lowest value exclude nothing, so that their sum stays above minus infinity; what
// ends there as one value is near, and told apart in FP64.
__device__ __forceinline__ float group_score(float a, float b)
{
    return b == -INFINITY ? a : fmaxf(a + b, -FLT_MAX);
}

// Routes one token with one warp, however close its values are.
template <int V, typename T>
__device__ __noinline__ void route_slowly(const RouteParams &p, int t, float bias_max, int *count, int lane)
{
    const T *row = static_cast<const T *>(p.logits) + static_cast<long long>(t) * p.ld;
    bool odd = false;
    float top = -INFINITY;
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 32 + lane;
        x[j] = e < p.experts ? to_float(row[e]) : -INFINITY;
        odd |= x[j] != x[j];
        top = fmaxf(top, x[j]);
    }
    const bool scored = p.bias != nullptr || p.groups > 1;
    float sum = 0.0f;
    if (!p.sigmoid) {
        top = warp_max(top);
        odd |= top == INFINITY;
        if (top == -INFINITY) top = 0.0f;
        if (scored || !p.renormalise) {
#pragma unroll 1
            for (int j = 0; j < V; ++j)
                if (j * 32 + lane < p.experts) sum += expf(to_float(row[j * 32 + lane]) - top);
            sum = warp_sum(sum);
        }
    }
    bool exactly = false;
    int index = -1;
    if (scored) {
        float most = 0.0f;
        uint32_t key[V];
        float score = -INFINITY;  // of group `lane`
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            float v = -INFINITY;
            if (x[j] != -INFINITY && e < p.experts) {
                const float s = p.sigmoid ? 1.0f / (1.0f + expf(-x[j])) : expf(x[j] - top) / sum;
                v = s + (p.bias ? __ldg(p.bias + e) : 0.0f);
                odd |= v != v;
                most = fmaxf(most, s);
            }
            x[j] = v;
            key[j] = key_of(v);
        }
        const float bound = score_bound(p, warp_max(most), bias_max);
        if (p.groups > 1) {
            for (int g = 0; g < p.groups; ++g) {
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if ((j * 32 + lane) / p.per_group == g) {
                        b = fmaxf(b, fminf(a, x[j]));
                        a = fmaxf(a, x[j]);
                    }
                warp_top2(a, b);
                if (lane == g) score = group_score(a, b);
            }
            uint32_t gkey[1] = {lane < p.groups ? key_of(score) : 0u}, mine;
            int open;
            pick<1>(gkey, p.top_groups + (p.top_groups < 32 ? 1 : 0), lane, mine, open);
            const float v = key_value(mine), next = __shfl_down_sync(kFull, v, 1);
            // the last group in and the first one out
            exactly |= lane == p.top_groups - 1 && lane < 31 && next != -INFINITY && !(v - next > 2.0f * bound);
            const uint32_t kept = __reduce_or_sync(kFull, open >= 0 && lane < p.top_groups ? 1u << open : 0u);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = j * 32 + lane;
                if (e < p.experts && !((kept >> (e / p.per_group)) & 1u)) key[j] = 0;
                if (!p.bias && key[j]) key[j] = key_of(to_float(row[e]));  // the ranking is the logits' own
            }
        }
        uint32_t mine;
        pick<V>(key, p.bias ? 32 : p.k, lane, mine, index);
        if (p.bias) {
            // The first 32 by FP32; the near ones among them settled in FP64.
            const float v = key_value(mine), next = __shfl_down_sync(kFull, v, 1);
            const bool close = lane < p.k && next != -INFINITY && !(v - next > bound);
            if (__any_sync(kFull, close)) {
                const float kth = __shfl_sync(kFull, v, p.k - 1), last = __shfl_sync(kFull, v, 31);
                if (!p.sigmoid || (last != -INFINITY && !(kth - last > bound))) {
                    exactly = true;
                } else {
                    const double d = index >= 0 ? 1.0 / (1.0 + exp(-static_cast<double>(to_float(row[index])))) +
                                                      static_cast<double>(__ldg(p.bias + index))
                                                : -INFINITY;
                    int rank = 0;
                    for (int i = 0; i < 32; ++i) {
                        const double o = __shfl_sync(kFull, d, i);
                        const int oi = __shfl_sync(kFull, index, i);
                        rank += o > d || (o == d && oi < index && oi >= 0) ? 1 : 0;
                    }
                    if (index < 0) rank = lane;  // these come last as they are
                    int found = -1;
                    for (int i = 0; i < 32; ++i) {
                        const int r = __shfl_sync(kFull, rank, i), oi = __shfl_sync(kFull, index, i);
                        if (r == lane) found = oi;
                    }
                    index = found;
                }
            }
        }
    } else {
        uint32_t key[V], unused;
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = key_of(x[j]);
        pick<V>(key, p.k, lane, unused, index);
    }
    float weight = __int_as_float(0x7fffffff);
    if (__any_sync(kFull, odd)) {
        index = -1;
    } else {
        if (__any_sync(kFull, exactly)) index = choose_exactly<V, T>(p, row, lane);
        if (lane >= p.k) index = -1;
        const float chosen = index >= 0 ? to_float(row[index]) : -INFINITY;
        float score = 0.0f;
        if (p.sigmoid) {
            if (index >= 0) score = 1.0f / (1.0f + expf(-chosen));
            if (p.renormalise) score /= warp_sum(score) + kTiny;
        } else if (p.renormalise) {
            const float m = warp_max(chosen);
            if (index >= 0) score = expf(chosen - m);
            const float total = warp_sum(score);
            if (index >= 0) score /= total;
        } else if (index >= 0) {
            score = expf(chosen - top) / sum;
        }
        weight = p.scale * score;
    }
    if (lane < p.k) {
        const long long at = static_cast<long long>(t) * p.k + lane;
        p.expert[at] = index;
        p.weights[at] = weight;
        atomicAdd(count + index + 1, 1);
    }
    __syncwarp();
}

// ------------------------------------------------------------ sorted key lists

__device__ __forceinline__ void order(uint32_t &a, uint32_t &b)  // the larger first
{
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}

// A bitonic list of eight, falling.
__device__ __forceinline__ void merge8(uint32_t (&a)[8])
{
#pragma unroll
    for (int d = 4; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order(a[i], a[i + d]);
}

__device__ __forceinline__ void sort8(uint32_t *a)  // odd-even merge sort
{
    order(a[0], a[1]), order(a[2], a[3]), order(a[4], a[5]), order(a[6], a[7]);
    order(a[0], a[2]), order(a[1], a[3]), order(a[4], a[6]), order(a[5], a[7]);
    order(a[1], a[2]), order(a[5], a[6]);
    order(a[0], a[4]), order(a[1], a[5]), order(a[2], a[6]), order(a[3], a[7]);
    order(a[2], a[4]), order(a[3], a[5]);
    order(a[1], a[2]), order(a[3], a[4]), order(a[5], a[6]);
}

// Where a lane's experts are: `lanes` lanes a group, `each` experts a lane.
struct Layout {
    int lanes, each;
    bool vec;  // 16-byte loads
};

template <int V>
__device__ __forceinline__ void load_row(const float *src, int n, bool vec, float (&x)[V])
{
    if (vec) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
            if (j < n) {
                const float4 v = *reinterpret_cast<const float4 *>(src + j);
                x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
            }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < n) x[j] = src[j];
    }
}

template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *src, int n, bool vec, float (&x)[V])
{
    if (vec) {
#pragma unroll
        for (int j = 0; j < V; j += 8)
            if (j < n) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[j + 2 * i] = __uint_as_float(w[i] << 16);
                    x[j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < n) x[j] = __bfloat162float(src[j]);
    }
}

// Within the L lanes of a token.
template <int L, typename F, typename Op>
__device__ __forceinline__ F token_reduce(F x, const Op &op)
{
#pragma unroll
    for (int d = L / 2; d; d >>= 1) x = op(x, __shfl_xor_sync(kFull, x, d));
    return x;
}

constexpr int kScratch = 32;  // candidates of settle_token, per warp
constexpr uint32_t kIndex = 511;            // the index in a key of an FP32 value
constexpr uint32_t kLowest = 0x00800000u;  // key of the lowest finite value, its index cut off

// The choice among n <= 32 experts of token t (scratch[0 .. n - 1]), the only ones
// that may be chosen, by logits or by sigmoid scores with a bias, in FP64 where
// two are within `bound`.  top, sum: of the row's softmax.
template <typename T>
__device__ __noinline__ void settle_token(const RouteParams &p, int t, int n, const int *scratch, float top, float sum,
                                          float bound, int *count, int lane)
{
    const T *row = static_cast<const T *>(p.logits) + static_cast<long long>(t) * p.ld;
    const int index = lane < n ? scratch[lane] : -1;
    const float x = index >= 0 ? to_float(row[index]) : -INFINITY;
    const float v = p.bias && index >= 0 ? 1.0f / (1.0f + expf(-x)) + __ldg(p.bias + index) : x;
    int rank = 0;
    bool close = false;
    for (int i = 0; i < n; ++i) {
        const float o = __shfl_sync(kFull, v, i);
        const int oi = __shfl_sync(kFull, index, i);
        rank += o > v || (o == v && oi < index) ? 1 : 0;
        close |= i != lane && !(fabsf(o - v) > bound);
    }
    if (p.bias && __any_sync(kFull, close && index >= 0)) {
        double d = -INFINITY;
        if (index >= 0) d = 1.0 / (1.0 + exp(-static_cast<double>(x))) + static_cast<double>(__ldg(p.bias + index));
        rank = 0;
        for (int i = 0; i < n; ++i) {
            const double o = __shfl_sync(kFull, d, i);
            const int oi = __shfl_sync(kFull, index, i);
            rank += o > d || (o == d && oi < index) ? 1 : 0;
        }
    }
    const bool in = index >= 0 && rank < p.k;
    float score = 0.0f;
    if (p.sigmoid) {
        if (in) score = 1.0f / (1.0f + expf(-x));
        if (p.renormalise) score /= warp_sum(score) + kTiny;
    } else if (p.renormalise) {
        const float m = warp_max(in ? x : -INFINITY);
        if (in) score = expf(x - m);
        score /= warp_sum(score);
    } else if (in) {
        score = expf(x - top) / sum;
    }
    if (in) {  // all k choices are there: one that is not would have ended the search
        const long long at = static_cast<long long>(t) * p.k + rank;
        p.expert[at] = index;
        p.weights[at] = p.scale * score;
        atomicAdd(count + index + 1, 1);
    }
}

// Routes tokens t0 + (lane / L), of which those below t1 are there.
template <int L, int V, typename T>
__device__ __forceinline__ void route_tokens(const RouteParams &p, const Layout &y, int t0, int t1, float bias_max,
                                             const float *bias, int *count, int *scratch, int lane)
{
    constexpr bool WHOLE_KEY = sizeof(T) == 2;  // without a bias: 16 bits of value, 16 of index
    const auto fmax_ = [](float a, float b) { return fmaxf(a, b); };
    const auto add = [](float a, float b) { return a + b; };
    const int ll = lane % L, t = t0 + lane / L;
    const unsigned token_mask = (L == 32 ? kFull : (1u << L) - 1u) << (lane / L * L);
    const int group = ll / y.lanes, sub = ll % y.lanes;
    const int first = group * p.per_group + sub * y.each;
    const int n = t < t1 && group < p.groups ? max(0, min(y.each, p.per_group - sub * y.each)) : 0;
    const T *row = static_cast<const T *>(p.logits) + static_cast<long long>(t) * p.ld;
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = -INFINITY;
    load_row<V>(row + first, n, y.vec, x);
    bool odd = false;
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j >= n) x[j] = -INFINITY;  // a 16-byte load may reach past
        odd |= x[j] != x[j];
        top = fmaxf(top, x[j]);
    }
    const bool biased = p.bias != nullptr, scored = biased || p.groups > 1;
    const bool whole_key = WHOLE_KEY && !biased;
    float sum = 0.0f;
    if (!p.sigmoid) {
        top = token_reduce<L>(top, fmax_);
        odd |= top == INFINITY;
        if (top == -INFINITY) top = 0.0f;
        if (scored || !p.renormalise) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(x[j] - top);
            sum = token_reduce<L>(sum, add);
        }
    }
    uint32_t key[V];
    bool close = false, open = true, slow_group = false;
    float bound = 0.0f, rough = 0.0f;  // of scores by expf, and of v
    if (scored) {
        float most = 0.0f, v[V], offset[V];
        const float scale = 1.0f / sum;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 b = biased ? *reinterpret_cast<const float4 *>(bias + ll * V + j) : make_float4(0, 0, 0, 0);
            offset[j] = b.x, offset[j + 1] = b.y, offset[j + 2] = b.z, offset[j + 3] = b.w;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float s = p.sigmoid ? inverse_near(1.0f + exp_near(-x[j])) : exp_near(x[j] - top) * scale;
            v[j] = x[j] == -INFINITY ? -INFINITY : s + offset[j];
            odd |= v[j] != v[j];
            if (x[j] != -INFINITY) most = fmaxf(most, s);
        }
        most = token_reduce<L>(most, fmax_);
        bound = score_bound(p, most, bias_max);
        // two scores by exp_near: (|x| + 7) 2^-24 of a sigmoid each, |x| up to 88
        rough = bound + most * (p.sigmoid ? 1.2e-5f : 1e-6f);
        if (p.groups > 1) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                b = fmaxf(b, fminf(a, v[j]));
                a = fmaxf(a, v[j]);
            }
            for (int d = y.lanes >> 1; d; d >>= 1) {
                const float a2 = __shfl_xor_sync(kFull, a, d), b2 = __shfl_xor_sync(kFull, b, d);
                b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                a = fmaxf(a, a2);
            }
            const float score = group_score(a, b);
            int rank = 0;
            bool near = false;
            for (int g = 0; g < p.groups; ++g) {
                const float o = __shfl_sync(kFull, score, (lane / L) * L + g * y.lanes);
                rank += o > score || (o == score && g < group) ? 1 : 0;
                near |= g != group && !(fabsf(o - score) > 2.0f * rough) && o != -INFINITY;
            }
            open = rank < p.top_groups && score != -INFINITY;
            // the last group in and the first one out may change places
            near = near && score != -INFINITY && (rank == p.top_groups - 1 || rank == p.top_groups);
            if (!p.sigmoid) {
                slow_group = near;
            } else if (__any_sync(kFull, near)) {
                // the sums again in FP64, of all that may be a group's two best
                const float least = (b == -INFINITY ? a : b) - rough;
                uint32_t which = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) which |= v[j] != -INFINITY && v[j] >= least ? 1u << j : 0u;
                double da = -INFINITY, db = -INFINITY;
                while (__any_sync(kFull, which != 0)) {
                    if (which != 0) {
                        const int j = __ffs(static_cast<int>(which)) - 1;
                        which &= which - 1;
                        const double d = 1.0 / (1.0 + exp(-static_cast<double>(to_float(row[first + j])))) +
                                         (biased ? static_cast<double>(__ldg(p.bias + first + j)) : 0.0);
                        if (d > da) {
                            db = da;
                            da = d;
                        } else if (d > db) {
                            db = d;
                        }
                    }
                    __syncwarp();
                }
                __syncwarp();
                for (int d = y.lanes >> 1; d; d >>= 1) {
                    const double a2 = __shfl_xor_sync(kFull, da, d), b2 = __shfl_xor_sync(kFull, db, d);
                    const double low = da < a2 ? da : a2, best = db < b2 ? b2 : db;
                    db = low < best ? best : low;
                    da = da < a2 ? a2 : da;
                }
                const double exact = db == -INFINITY ? da : da + db;
                rank = 0;
                for (int g = 0; g < p.groups; ++g) {
                    const double o = __shfl_sync(kFull, exact, (lane / L) * L + g * y.lanes);
                    rank += o > exact || (o == exact && g < group) ? 1 : 0;
                }
                open = rank < p.top_groups && score != -INFINITY;
            }
        }
        if (biased)
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = v[j];
    }
    // Minus infinity, what is past the row's end and closed groups come out below
    // kLowest, the key of the lowest finite value.
    const uint32_t keep = open ? (whole_key ? 0xffff0000u : ~kIndex) : 0u;
    const uint32_t base = (whole_key ? 0xffffu : kIndex) - static_cast<uint32_t>(first);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t u = __float_as_uint(x[j] + 0.0f);
        key[j] = ((u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u)) & keep) |
                 ((base - j) & (whole_key ? 0xffffu : kIndex));
    }
    uint32_t list[8];
    if (V == 16) {
        uint32_t other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            list[i] = key[i];
            other[i] = key[V - 8 + i];
        }
        sort8(list);
        sort8(other);
#pragma unroll
        for (int i = 0; i < 8; ++i) list[i] = max(list[i], other[7 - i]);
        merge8(list);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) list[i] = key[i];
        sort8(list);
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) {
        uint32_t other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kFull, list[7 - i], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) list[i] = max(list[i], other[i]);
        merge8(list);
    }
    uint32_t mine = 0, last = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i == ll) mine = list[i];
        if (i == p.k - 1) last = list[i];
    }
    if (ll >= p.k) mine = 0;
    const bool full = last >= kLowest;  // k choices
    uint32_t low = kLowest;
    if (!whole_key && full) {
        // whatever is not chosen and may belong before the last choice
        low = last & ~kIndex;
        if (biased) low = min(low, key_of(key_value(low) - rough) & ~kIndex);
        low = max(low, kLowest);
#pragma unroll
        for (int j = 0; j < V; ++j) close |= key[j] < last && key[j] >= low;
    }
    const int index = mine < kLowest ? -1 : static_cast<int>(whole_key ? 0xffffu - (mine & 0xffffu) : kIndex - (mine & kIndex));
    const float chosen = index >= 0 ? to_float(row[index]) : -INFINITY;
    float score = 0.0f;
    if (p.sigmoid) {
        if (index >= 0) score = 1.0f / (1.0f + expf(-chosen));
    }
    int rank = ll;
    if (!whole_key) {
        const float v = biased ? (index >= 0 ? (p.sigmoid ? score : expf(chosen - top) / sum) + __ldg(p.bias + index) : -INFINITY)
                               : chosen;
        int before = 0;
        for (int i = 0; i < p.k; ++i) {
            const float o = __shfl_sync(kFull, v, (lane / L) * L + i);
            const int oi = __shfl_sync(kFull, index, (lane / L) * L + i);
            before += oi >= 0 && (o > v || (o == v && oi < index)) ? 1 : 0;
            close |= biased && index >= 0 && oi >= 0 && oi != index && !(fabsf(o - v) > bound);
        }
        if (index >= 0) rank = before;
    }
    if (p.sigmoid) {
        if (p.renormalise) score /= token_reduce<8>(score, add) + kTiny;
    } else if (p.renormalise) {
        const float m = token_reduce<8>(chosen, fmax_);
        if (index >= 0) score = expf(chosen - m);
        const float total = token_reduce<8>(score, add);
        if (index >= 0) score /= total;
    } else if (index >= 0) {
        score = expf(chosen - top) / sum;
    }
    const bool bad = (__ballot_sync(kFull, odd) & token_mask) != 0;
    // A softmax with a bias needs the whole row in FP64.
    const unsigned again = __ballot_sync(kFull, (slow_group || (close && biased && !p.sigmoid)) && !bad && t < t1);
    const unsigned unsettled = __ballot_sync(kFull, close && !bad && t < t1) | again;
    if (ll < p.k && t < t1 && (unsettled & token_mask) == 0) {
        const long long at = static_cast<long long>(t) * p.k + (bad ? ll : rank);
        p.expert[at] = bad ? -1 : index;
        p.weights[at] = bad ? __int_as_float(0x7fffffff) : p.scale * score;
        atomicAdd(count + (bad ? 0 : index + 1), 1);
    }
    if (unsettled == 0) return;
    for (int i = 0; i < 32 / L; ++i) {
        const unsigned mask = (L == 32 ? kFull : (1u << L) - 1u) << (i * L);
        if ((unsettled & mask) == 0) continue;
        // how many experts may be among the chosen, and which
        int mine_n = 0;
        if (lane / L == i)
#pragma unroll
            for (int j = 0; j < V; ++j) mine_n += key[j] >= low ? 1 : 0;
        int at = mine_n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(kFull, at, d);
            if (lane >= d) at += up;
        }
        const int n = __shfl_sync(kFull, at, 31);
        // without a last choice nothing was cut off, and only a warp's own pick
        // knows how many there are
        const bool few = n <= kScratch && __shfl_sync(kFull, full ? 1 : 0, i * L) != 0;
        if ((again & mask) != 0 || !few) {
            route_slowly<16, T>(p, t0 + i, bias_max, count, lane);
            continue;
        }
        at -= mine_n;
        if (lane / L == i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] >= low) scratch[at++] = first + j;
        __syncwarp();
        settle_token<T>(p, t0 + i, n, scratch, __shfl_sync(kFull, top, i * L), __shfl_sync(kFull, sum, i * L),
                        __shfl_sync(kFull, bound, i * L), count, lane);
        __syncwarp();
    }
}

// Exclusive prefix sums of v[0 .. n - 1] in place; every thread of the CTA.
template <int NT>
__device__ void block_scan(int *v, int n, int *warp_sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + NT - 1) / NT;
    const int lo = min(n, tid * per), hi = min(n, lo + per);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += v[i];
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFull, inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    for (int i = lo; i < hi; ++i) {
        const int x = v[i];
        v[i] = before;
        before += x;
    }
    __syncthreads();
}

// A warp's run of the choices lo .. hi - 1 (rows t * k + i), whole 32s, and the bins
// (expert + 1) of its first KEEP * 32, a lane's own.
template <int NT>
struct Run {
    static constexpr int KEEP = 4;
    int first, last, bin[KEEP];
    __device__ __forceinline__ void load(const RouteParams &p, int lo, int hi)
    {
        constexpr int W = NT / 32;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = ((hi - lo + W - 1) / W + 31) & ~31;
        first = lo + warp * per;
        last = min(hi, first + per);
#pragma unroll
        for (int j = 0; j < KEEP; ++j) bin[j] = at(p, first + j * 32 + lane);
    }
    __device__ __forceinline__ int at(const RouteParams &p, int i) const
    {
        return i < last ? static_cast<int>(p.expert[i]) + 1 : -1;
    }
};

// Places the choices of all warps' runs by expert.  base[b]: where the first of bin
// b goes.  hist: [warps][bins] of zeros.
template <int NT>
__device__ void place(const RouteParams &p, const Run<NT> &run, int bins, const int *base, int *hist)
{
    constexpr int W = NT / 32, KEEP = Run<NT>::KEEP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *mine = hist + warp * bins;
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
        if (run.bin[j] >= 0) atomicAdd(mine + run.bin[j], 1);
    for (int i = run.first + KEEP * 32 + lane; i < run.last; i += 32) atomicAdd(mine + run.at(p, i), 1);
    __syncthreads();
    for (int b = tid; b < bins; b += NT) {
        int at = base[b];
#pragma unroll 8
        for (int w = 0; w < W; ++w) {
            const int n = hist[w * bins + b];
            hist[w * bins + b] = at;
            at += n;
        }
    }
    __syncthreads();
    const auto put = [&](int i, int bin) {
        const unsigned same = __match_any_sync(kFull, bin);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int at = bin >= 0 ? mine[bin] : 0;
        __syncwarp();
        if (bin >= 0) {
            if (rank == 0) mine[bin] = at + __popc(same);
            p.order[at + rank] = i;
        }
        __syncwarp();
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
        if (run.first + j * 32 < run.last) put(run.first + j * 32 + lane, run.bin[j]);
    for (int i0 = run.first + KEEP * 32; i0 < run.last; i0 += 32) put(i0 + lane, run.at(p, i0 + lane));
}

__device__ __forceinline__ float largest_bias(const RouteParams &p, int lane)
{
    float m = 0.0f;
    if (p.bias)
        for (int e = lane; e < p.experts; e += 32) {
            const float b = fabsf(__ldg(p.bias + e));
            if (b < INFINITY) m = fmaxf(m, b);
        }
    return warp_max(m);
}

// L lanes a token with V experts each; L = 0: every token by route_slowly, V * 32
// experts at most.  ONE: a single CTA, which also places.
template <int L, int V, int NT, typename T, bool ONE>
__global__ void __launch_bounds__(NT, 1) route_kernel(const RouteParams p, const Layout y)
{
    constexpr int W = NT / 32;
    extern __shared__ int smem[];
    __shared__ int warp_sums[W], scratch[W][kScratch];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = p.experts + 1;
    int *count = smem, *hist = smem + bins;  // ONE: a counter a warp and bin
    for (int i = tid; i < (ONE ? bins * (1 + W) : bins); i += NT) smem[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const float bias_max = largest_bias(p, lane);
    const int t0 = blockIdx.x * p.per_chunk, t1 = min(p.tokens, t0 + p.per_chunk);
    if constexpr (L > 0) {
        __shared__ __align__(16) float bias[L * V];  // as the lanes hold the experts
        if (p.bias) {
            for (int i = tid; i < L * V; i += NT) {
                const int l = i / V, j = i % V, group = l / y.lanes, at = l % y.lanes * y.each + j;
                const bool there = group < p.groups && j < y.each && at < p.per_group;
                bias[i] = there ? __ldg(p.bias + group * p.per_group + at) : 0.0f;
            }
            __syncthreads();
        }
        for (int t = t0 + warp * (32 / L); t < t1; t += W * (32 / L))
            route_tokens<L, V, T>(p, y, t, t1, bias_max, bias, count, scratch[warp], lane);
    } else {
        for (int t = t0 + warp; t < t1; t += W) route_slowly<V, T>(p, t, bias_max, count, lane);
    }
    __syncthreads();
    if (ONE) {
        block_scan<NT>(count, bins, warp_sums);
        for (int b = tid; b < bins; b += NT)  // bin e + 1 starts where expert e does
            if (b > 0) p.offsets[b - 1] = count[b];
        if (tid == 0) p.offsets[p.experts] = static_cast<long long>(p.tokens) * p.k;
        Run<NT> run;
        run.load(p, 0, p.tokens * p.k);
        place<NT>(p, run, bins, count, hist);
    } else {
        for (int b = tid; b < p.pitch; b += NT)
            p.counts[static_cast<long long>(blockIdx.x) * p.pitch + b] = b < bins ? count[b] : 0;
    }
}

// The counts' rows are `pitch` long, whole 16 bytes.
template <int NT>
__global__ void __launch_bounds__(NT, 1) place_kernel(const RouteParams p)
{
    extern __shared__ int smem[];
    __shared__ int warp_sums[NT / 32];
    const int tid = threadIdx.x;
    const int bins = p.experts + 1;
    int *total = smem, *before = smem + bins, *hist = smem + 2 * bins;
    for (int i = tid; i < (2 + NT / 32) * bins; i += NT) smem[i] = 0;
    const int t0 = blockIdx.x * p.per_chunk, t1 = min(p.tokens, t0 + p.per_chunk);
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    Run<NT> run;
    run.load(p, t0 * p.k, max(t0, t1) * p.k);
    // four bins a thread, as many runs of CTAs side by side as there are threads
    const int quads = p.pitch / 4, parts = NT / quads;
    if (tid < parts * quads) {
        const int quad = tid % quads;
        int all[4] = {}, mine[4] = {};
#pragma unroll 8
        for (int c = tid / quads; c < p.chunks; c += parts) {
            const int4 n = *reinterpret_cast<const int4 *>(p.counts + static_cast<long long>(c) * p.pitch + quad * 4);
            const int v[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all[i] += v[i];
                if (c < static_cast<int>(blockIdx.x)) mine[i] += v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (quad * 4 + i < bins) {
                atomicAdd(total + quad * 4 + i, all[i]);
                atomicAdd(before + quad * 4 + i, mine[i]);
            }
    }
    __syncthreads();
    block_scan<NT>(total, bins, warp_sums);
    if (blockIdx.x == 0) {
        for (int b = tid; b < bins; b += NT)
            if (b > 0) p.offsets[b - 1] = total[b];
        if (tid == 0) p.offsets[p.experts] = static_cast<long long>(p.tokens) * p.k;
    }
    for (int b = tid; b < bins; b += NT) before[b] += total[b];
    __syncthreads();
    place<NT>(p, run, bins, before, hist);
}

__global__ void zero_offsets_kernel(long long *offsets, int n)
{
    for (int i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

// 64 registers a thread: route_kernel is bound by the latency of what a warp does
// (loads, exchanges), so that more warps win over more registers.
constexpr int NT = 1024;
constexpr size_t MOST_BINS = GEMM_ROUTE_MAX_EXPERTS + 1;

// A counter a warp and bin.
constexpr size_t hist_bytes(int threads, size_t bins) { return threads / 32 * bins * 4; }

template <int L, int V, typename T>
cudaError_t launch_typed(const RouteParams &p, const Layout &y, cudaStream_t stream, int *launches)
{
    const size_t bins = static_cast<size_t>(p.experts) + 1, hist = hist_bytes(NT, bins);
    cudaError_t e;
    if (p.chunks == 1) {
        e = kernel_ready<route_kernel<L, V, NT, T, true>>(MOST_BINS * 4 + hist_bytes(NT, MOST_BINS));
        if (e == cudaSuccess)
            e = launch_pdl(route_kernel<L, V, NT, T, true>, 1, NT, bins * 4 + hist, stream, 1, p, y);
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    e = kernel_ready<route_kernel<L, V, NT, T, false>>(0);
    if (e == cudaSuccess) e = kernel_ready<place_kernel<NT>>(2 * MOST_BINS * 4 + hist_bytes(NT, MOST_BINS));
    if (e == cudaSuccess) e = launch_pdl(route_kernel<L, V, NT, T, false>, p.chunks, NT, bins * 4, stream, 1, p, y);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_pdl(place_kernel<NT>, p.chunks, NT, 2 * bins * 4 + hist, stream, 1, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

template <typename T>
cudaError_t launch_for(const RouteParams &p, cudaStream_t stream, int *launches)
{
    if (p.k <= 8)
        for (int L = 8; L <= 32; L *= 2) {
            // the fewest lanes that hold the experts, whole groups each
            Layout y;
            y.lanes = L;
            while (y.lanes * p.groups > L && y.lanes > 0) y.lanes >>= 1;
            if (y.lanes == 0) continue;
            const int vec = 16 / sizeof(T);
            y.each = (p.per_group + y.lanes - 1) / y.lanes;
            if (y.each > 16) continue;
            const int round = (y.each + vec - 1) / vec * vec;  // whole 16-byte pieces a lane where rows allow them
            y.vec = p.per_group % vec == 0 && p.ld % vec == 0 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
            if (y.vec) y.each = round;
            const bool small = y.each <= 8;
            if (L == 8) return small ? launch_typed<8, 8, T>(p, y, stream, launches) : launch_typed<8, 16, T>(p, y, stream, launches);
            if (L == 16) return small ? launch_typed<16, 8, T>(p, y, stream, launches) : launch_typed<16, 16, T>(p, y, stream, launches);
            return small ? launch_typed<32, 8, T>(p, y, stream, launches) : launch_typed<32, 16, T>(p, y, stream, launches);
        }
    const Layout none = {};
    return p.experts <= 512 ? launch_typed<0, 16, T>(p, none, stream, launches)
                            : launch_typed<0, 32, T>(p, none, stream, launches);
}

// ------------------------------------------------------------------ gradient

struct GradParams {
    const void *logits;
    long long ld;
    int tokens, experts, k;
    const long long *expert;
    const float *dweights;
    int sigmoid, renormalise;
    float scale;
    void *dlogits;
    long long ldd;
};

constexpr int GRAD_THREADS = 256;

__device__ __forceinline__ void store(float *out, float x) { *out = x; }
__device__ __forceinline__ void store(__nv_bfloat16 *out, float x) { *out = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store4(float *out, float4 x) { *reinterpret_cast<float4 *>(out) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *out, float4 x)
{
    const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
    *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(w);
}

// One warp a token: the chosen experts' derivatives are put into a row of
// zeros in shared memory, which goes out whole.  VEC: elements a lane writes at
// once (4 where the rows of dlogits start on its boundaries, else 1).
template <typename T, int VEC>
__global__ void __launch_bounds__(GRAD_THREADS) route_grad_kernel(const GradParams p)
{
    extern __shared__ float rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wide = (p.experts + 3) & ~3;
    float *row = rows + warp * wide;
    for (int e = lane; e < wide; e += 32) row[e] = 0.0f;
    __syncwarp();
    griddep_wait();
    griddep_launch_dependents();
    const bool whole = !p.sigmoid && !p.renormalise;
    for (int t = blockIdx.x * (GRAD_THREADS / 32) + warp; t < p.tokens; t += gridDim.x * (GRAD_THREADS / 32)) {
        const T *x = static_cast<const T *>(p.logits) + static_cast<long long>(t) * p.ld;
        T *out = static_cast<T *>(p.dlogits) + static_cast<long long>(t) * p.ldd;
        int index = -1;
        float g = 0.0f, chosen = -INFINITY;
        if (lane < p.k) {
            const long long at = static_cast<long long>(t) * p.k + lane;
            const long long e = p.expert[at];
            if (e >= 0 && e < p.experts) {
                index = static_cast<int>(e);
                g = p.dweights[at] * p.scale;
                chosen = to_float(x[index]);
            }
        }
        const bool any = __any_sync(kFull, index >= 0);
        float value = 0.0f, top = 0.0f, inv = 0.0f, dot = 0.0f;
        if (whole && any) {
            float m = -INFINITY, s = 0.0f;  // running maximum and sum
            for (int e = lane; e < p.experts; e += 32) {
                const float v = to_float(x[e]);
                const float n = fmaxf(m, v);
                if (n != -INFINITY) s = s * expf(m - n) + expf(v - n);
                m = n;
            }
            top = warp_max(m);
            s = warp_sum(m == -INFINITY ? 0.0f : s * expf(m - top));
            inv = 1.0f / s;
            value = index >= 0 ? expf(chosen - top) * inv * g : 0.0f;
            dot = warp_sum(value);
        } else if (!p.sigmoid) {
            const float m = warp_max(chosen);
            const float e = index >= 0 ? expf(chosen - m) : 0.0f;
            const float total = warp_sum(e);
            const float w = index >= 0 ? e / total : 0.0f;
            value = w * (g - warp_sum(w * g));
        } else {
            const float s = index >= 0 ? 1.0f / (1.0f + expf(-chosen)) : 0.0f;
            if (p.renormalise) {
                const float total = warp_sum(s) + kTiny;
                g = (g - warp_sum(s / total * g)) / total;
            }
            // 1 - sigmoid(x) = sigmoid(-x), without the cancellation
            if (index >= 0) value = g * s / (1.0f + expf(chosen));
        }
        if (index >= 0) atomicAdd(row + index, value);
        __syncwarp();
        if (VEC == 4) {
            for (int e = lane * 4; e < p.experts; e += 128) {
                float4 v = *reinterpret_cast<const float4 *>(row + e);
                if (whole && any) {
                    v.x -= expf(to_float(x[e]) - top) * inv * dot;
                    v.y -= expf(to_float(x[e + 1]) - top) * inv * dot;
                    v.z -= expf(to_float(x[e + 2]) - top) * inv * dot;
                    v.w -= expf(to_float(x[e + 3]) - top) * inv * dot;
                }
                store4(out + e, v);
            }
        } else {
            for (int e = lane; e < p.experts; e += 32) {
                float v = row[e];
                if (whole && any) v -= expf(to_float(x[e]) - top) * inv * dot;
                store(out + e, v);
            }
        }
        __syncwarp();
        if (index >= 0) row[index] = 0.0f;
        __syncwarp();
    }
}

template <typename T>
cudaError_t launch_grad(const RouteGradArgs &a, const GradParams &p, int sm_count, int max_ctas)
{
    const bool vec = p.experts % 4 == 0 && p.ldd % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % (4 * sizeof(T)) == 0;
    const int warps = GRAD_THREADS / 32;
    const size_t smem = static_cast<size_t>(warps) * ((p.experts + 3) & ~3) * 4;
    const int grid = capped(std::min((p.tokens + warps - 1) / warps, 8 * sm_count), max_ctas);
    const cudaError_t e = vec ? kernel_ready<route_grad_kernel<T, 4>>(0) : kernel_ready<route_grad_kernel<T, 1>>(0);
    if (e != cudaSuccess) return e;
    return vec ? launch_pdl(route_grad_kernel<T, 4>, grid, GRAD_THREADS, smem, a.stream, 1, p)
               : launch_pdl(route_grad_kernel<T, 1>, grid, GRAD_THREADS, smem, a.stream, 1, p);
}

}  // namespace

static int count_pitch(int64_t experts) { return static_cast<int>((experts + 1 + 3) / 4 * 4); }

int route_chunks(int64_t tokens, int sm_count)
{
    // one CTA up to 64 tokens: it also sorts, without a second launch
    if (tokens <= 64) return 1;
    return static_cast<int>(std::min<int64_t>((tokens + 31) / 32, sm_count));
}

size_t route_workspace(int64_t tokens, int64_t experts, int sm_count)
{
    const int chunks = route_chunks(tokens, sm_count);
    return chunks == 1 ? 0 : static_cast<size_t>(chunks) * count_pitch(experts) * 4;
}

cudaError_t launch_route(const RouteArgs &a, int sm_count, int *launches)
{
    if (a.tokens == 0) {
        zero_offsets_kernel<<<1, 256, 0, a.stream>>>(a.offsets, a.experts + 1);
        const cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    RouteParams p;
    p.logits = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.experts = a.experts;
    p.k = a.k;
    p.bias = a.bias;
    p.groups = a.groups;
    p.top_groups = a.top_groups;
    p.per_group = a.experts / a.groups;
    p.sigmoid = a.sigmoid;
    p.renormalise = a.renormalise;
    p.scale = a.scale;
    p.weights = a.weights;
    p.expert = a.expert;
    p.order = a.order;
    p.offsets = a.offsets;
    p.counts = a.counts;
    p.chunks = route_chunks(a.tokens, sm_count);
    p.per_chunk = (a.tokens + p.chunks - 1) / p.chunks;
    p.pitch = count_pitch(a.experts);
    return a.bf16 ? launch_for<__nv_bfloat16>(p, a.stream, launches) : launch_for<float>(p, a.stream, launches);
}

cudaError_t launch_route_grad(const RouteGradArgs &a, int sm_count, int max_ctas)
{
    GradParams p;
    p.logits = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.experts = a.experts;
    p.k = a.k;
    p.expert = a.expert;
    p.dweights = a.dweights;
    p.sigmoid = a.sigmoid;
    p.renormalise = a.renormalise;
    p.scale = a.scale;
    p.dlogits = a.dlogits;
    p.ldd = a.ldd;
    return a.bf16 ? launch_grad<__nv_bfloat16>(a, p, sm_count, max_ctas)
                  : launch_grad<float>(a, p, sm_count, max_ctas);
}

}  // namespace dg
