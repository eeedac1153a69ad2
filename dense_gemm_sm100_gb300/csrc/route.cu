// Routing of tokens to experts: scores, the k best experts of every token with
// their weights, the rows sorted by expert with the experts' offsets, and the
// gradient of the logits.
//
// One warp a token.  Lane l holds the logits of experts l, l + 32, ...; a pick
// is a warp-wide maximum of order-preserving integer keys (redux.sync), then
// the lowest index that has it, and lane i keeps pick i.  Two values that FP32
// cannot tell apart (closer than a bound on the rounding of the scores) send
// the warp through the same choice in FP64; without a bias or groups the
// logits themselves are compared and nothing is ever close.
//
// Sorting by expert is a counting sort, stable and without atomics whose order
// would matter: CTA c routes a run of tokens and counts its choices by expert;
// a second launch adds the counts of the CTAs before it, and places its own
// run, warp by warp, with a warp-wide match for the rank among 32 choices.
// Where one CTA does all tokens, both steps are one launch.
#include <cuda_bf16.h>

#include <algorithm>
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

// The choice of a row in FP64, with a bias or groups: lane i < k gets pick i.
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
            for (int d = 16; d; d >>= 1) {
                const double a2 = __shfl_xor_sync(kFull, a, d), b2 = __shfl_xor_sync(kFull, b, d);
                b = fmax(fmin(a, a2), fmax(b, b2));
                a = fmax(a, a2);
            }
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

// Routes token t with one warp: lane i < k gets choice i (-1: none) and its
// weight.  x: the row (minus infinity past its end).
template <int V, typename T>
__device__ __forceinline__ int route_row(const RouteParams &p, const T *row, const float (&x)[V], float bias_max,
                                         float *scratch, int lane, float &weight)
{
    bool odd = false;
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        odd |= x[j] != x[j];
        top = fmaxf(top, x[j]);
    }
    const bool scored = p.bias != nullptr || p.groups > 1;
    const bool whole = !p.sigmoid && (scored || !p.renormalise);  // the softmax's sum is needed
    float sum = 0.0f;
    if (!p.sigmoid) {
        top = warp_max(top);
        odd |= top == INFINITY;
        if (top == -INFINITY) top = 0.0f;
        if (whole) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(x[j] - top);
            sum = warp_sum(sum);
        }
    }
    uint32_t key[V];
    bool close = false;
    float bound = 0.0f;  // on how far two of the compared values may be off
    if (scored) {
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            const float s = p.sigmoid ? 1.0f / (1.0f + expf(-x[j])) : expf(x[j] - top) / sum;
            const float b = p.bias && e < p.experts ? __ldg(p.bias + e) : 0.0f;
            const float v = x[j] == -INFINITY ? -INFINITY : s + b;
            odd |= v != v;
            if (x[j] != -INFINITY) most = fmaxf(most, s);
            key[j] = key_of(v);
            if (p.groups > 1 && e < p.experts) scratch[e + e / p.per_group] = v;
        }
        // FP32 exp, sum, division and the bias's addition stay within 2^-18 of these
        bound = (warp_max(most) + bias_max) * 4e-6f;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = key_of(x[j]);
    }
    if (__any_sync(kFull, odd)) {
        weight = __int_as_float(0x7fffffff);
        return -1;
    }
    if (p.groups > 1) {
        __syncwarp();
        // `lanes` lanes a group find its two best
        int lanes = 32;
        while (lanes * p.groups > 32) lanes >>= 1;
        const int g = lane / lanes;
        float a = -INFINITY, b = -INFINITY;
        if (g < p.groups)
            for (int i = lane % lanes; i < p.per_group; i += lanes) {
                const float v = scratch[g * (p.per_group + 1) + i];
                b = fmaxf(b, fminf(a, v));
                a = fmaxf(a, v);
            }
        for (int d = lanes >> 1; d; d >>= 1) {
            const float a2 = __shfl_xor_sync(kFull, a, d), b2 = __shfl_xor_sync(kFull, b, d);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        }
        // group g's score in lane g
        const float score = __shfl_sync(kFull, b == -INFINITY ? a : a + b, (lane * lanes) & 31);
        uint32_t gkey[1] = {lane < p.groups ? key_of(score) : 0u}, mine;
        int open;
        pick<1>(gkey, p.top_groups + (p.top_groups < 32 ? 1 : 0), lane, mine, open);
        const float v = key_value(mine), next = __shfl_down_sync(kFull, v, 1);
        // the last group in and the first one out
        close |= lane == p.top_groups - 1 && lane < 31 && next != -INFINITY && !(v - next > 2.0f * bound);
        const uint32_t kept = __reduce_or_sync(kFull, open >= 0 && lane < p.top_groups ? 1u << open : 0u);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            if (!p.bias) key[j] = key_of(x[j]);
            if (e < p.experts && !((kept >> (e / p.per_group)) & 1u)) key[j] = 0;
        }
    }
    uint32_t mine;
    int index;
    pick<V>(key, p.k + (p.bias ? 1 : 0), lane, mine, index);
    if (p.bias) {
        const float v = key_value(mine), next = __shfl_down_sync(kFull, v, 1);
        close |= lane < p.k && next != -INFINITY && !(v - next > bound);
    }
    if (scored && __any_sync(kFull, close)) index = choose_exactly<V, T>(p, row, lane);
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
    return index;
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

// Places the choices lo .. hi - 1 (rows t * k + i) by expert.  base[b]: where
// the first of bin b = expert + 1 goes.  hist: [warps][bins] of scratch.
template <int NT>
__device__ void place(const RouteParams &p, int lo, int hi, int bins, const int *base, int *hist)
{
    constexpr int W = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < W * bins; i += NT) hist[i] = 0;
    __syncthreads();
    // a contiguous run of whole 32s a warp
    const int per = ((hi - lo + W - 1) / W + 31) & ~31;
    const int first = lo + warp * per, last = min(hi, first + per);
    int *mine = hist + warp * bins;
    for (int i = first + lane; i < last; i += 32) atomicAdd(mine + static_cast<int>(p.expert[i]) + 1, 1);
    __syncthreads();
    for (int b = tid; b < bins; b += NT) {
        int at = base[b];
        for (int w = 0; w < W; ++w) {
            const int n = hist[w * bins + b];
            hist[w * bins + b] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int i0 = first; i0 < last; i0 += 32) {
        const int i = i0 + lane;
        const int bin = i < last ? static_cast<int>(p.expert[i]) + 1 : -1;
        const unsigned same = __match_any_sync(kFull, bin);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int at = bin >= 0 ? mine[bin] : 0;
        __syncwarp();
        if (bin >= 0) {
            if (rank == 0) mine[bin] = at + __popc(same);
            p.order[at + rank] = i;
        }
        __syncwarp();
    }
}

// ONE: a single CTA, which also places.
template <int V, int NT, typename T, bool ONE>
__global__ void __launch_bounds__(NT, 1) route_kernel(const RouteParams p)
{
    constexpr int W = NT / 32;
    extern __shared__ int smem[];
    __shared__ int warp_sums[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = p.experts + 1;
    int *count = smem, *hist = smem + bins;  // hist: ONE only; the warps' scratch overlays it
    float *scratch = reinterpret_cast<float *>(hist) + warp * (p.experts + p.groups);
    for (int i = tid; i < bins; i += NT) count[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    float bias_max = 0.0f;
    if (p.bias) {
        for (int e = lane; e < p.experts; e += 32) {
            const float b = fabsf(__ldg(p.bias + e));
            if (b < INFINITY) bias_max = fmaxf(bias_max, b);
        }
        bias_max = warp_max(bias_max);
    }
    const int t0 = blockIdx.x * p.per_chunk, t1 = min(p.tokens, t0 + p.per_chunk);
    const T *logits = static_cast<const T *>(p.logits);
    float next[V];
    const auto fetch = [&](int t) {
        const T *row = logits + static_cast<long long>(t) * p.ld;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            next[j] = t < t1 && e < p.experts ? to_float(row[e]) : -INFINITY;
        }
    };
    fetch(t0 + warp);
    for (int t = t0 + warp; t < t1; t += W) {
        float x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = next[j];
        fetch(t + W);
        float weight;
        const int index =
            route_row<V, T>(p, logits + static_cast<long long>(t) * p.ld, x, bias_max, scratch, lane, weight);
        if (lane < p.k) {
            const long long at = static_cast<long long>(t) * p.k + lane;
            p.expert[at] = index;
            p.weights[at] = weight;
            atomicAdd(count + index + 1, 1);
        }
        __syncwarp();
    }
    __syncthreads();
    if (ONE) {
        block_scan<NT>(count, bins, warp_sums);
        for (int b = tid; b < bins; b += NT)  // bin e + 1 starts where expert e does
            if (b > 0) p.offsets[b - 1] = count[b];
        if (tid == 0) p.offsets[p.experts] = static_cast<long long>(p.tokens) * p.k;
        place<NT>(p, 0, p.tokens * p.k, bins, count, hist);
    } else {
        for (int b = tid; b < bins; b += NT) p.counts[blockIdx.x * bins + b] = count[b];
    }
}

// V: the instance's most experts / 32, which its shared memory goes by.
template <int V, int NT>
__global__ void __launch_bounds__(NT, 1) place_kernel(const RouteParams p)
{
    extern __shared__ int smem[];
    __shared__ int warp_sums[NT / 32];
    const int tid = threadIdx.x;
    const int bins = p.experts + 1;
    int *total = smem, *before = smem + bins, *hist = smem + 2 * bins;
    for (int i = tid; i < 2 * bins; i += NT) smem[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    // whole warps of bins, so many runs of CTAs side by side
    const int wide = min(NT, (bins + 31) & ~31), parts = NT / wide;
    if (tid < parts * wide)
        for (int b = tid % wide; b < bins; b += wide) {
            int all = 0, mine = 0;
#pragma unroll 8
            for (int c = tid / wide; c < p.chunks; c += parts) {
                const int n = p.counts[c * bins + b];
                all += n;
                if (c < static_cast<int>(blockIdx.x)) mine += n;
            }
            atomicAdd(total + b, all);
            atomicAdd(before + b, mine);
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
    const int t0 = blockIdx.x * p.per_chunk, t1 = min(p.tokens, t0 + p.per_chunk);
    place<NT>(p, t0 * p.k, max(t0, t1) * p.k, bins, before, hist);
}

__global__ void zero_offsets_kernel(long long *offsets, int n)
{
    for (int i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

template <int V, int NT, typename T>
cudaError_t launch_typed(const RouteParams &p, cudaStream_t stream, int *launches)
{
    constexpr size_t W = NT / 32;
    const size_t bins = static_cast<size_t>(p.experts) + 1;
    const size_t scratch = p.groups > 1 ? W * (p.experts + p.groups) * 4 : 0, hist = W * bins * 4;
    // of the most experts these instances take
    constexpr size_t MOST_BINS = V * 32 + 1, MOST_HIST = W * (MOST_BINS + GEMM_ROUTE_MAX_GROUPS) * 4;
    cudaError_t e;
    if (p.chunks == 1) {
        e = kernel_ready<route_kernel<V, NT, T, true>>(MOST_BINS * 4 + MOST_HIST);
        if (e == cudaSuccess)
            e = launch_pdl(route_kernel<V, NT, T, true>, 1, NT, bins * 4 + std::max(scratch, hist), stream, 1, p);
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    e = kernel_ready<route_kernel<V, NT, T, false>>(MOST_BINS * 4 + MOST_HIST);
    if (e == cudaSuccess) e = kernel_ready<place_kernel<V, NT>>(2 * MOST_BINS * 4 + MOST_HIST);
    if (e == cudaSuccess)
        e = launch_pdl(route_kernel<V, NT, T, false>, p.chunks, NT, bins * 4 + scratch, stream, 1, p);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_pdl(place_kernel<V, NT>, p.chunks, NT, 2 * bins * 4 + hist, stream, 1, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

template <typename T>
cudaError_t launch_for(const RouteParams &p, cudaStream_t stream, int *launches)
{
    const int v = (p.experts + 31) / 32;
    if (v <= 1) return launch_typed<1, 1024, T>(p, stream, launches);
    if (v <= 2) return launch_typed<2, 1024, T>(p, stream, launches);
    if (v <= 4) return launch_typed<4, 1024, T>(p, stream, launches);
    if (v <= 8) return launch_typed<8, 1024, T>(p, stream, launches);
    if (v <= 16) return launch_typed<16, 512, T>(p, stream, launches);
    return launch_typed<32, 512, T>(p, stream, launches);
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
cudaError_t launch_grad(const RouteGradArgs &a, const GradParams &p, int sm_count)
{
    const bool vec = p.experts % 4 == 0 && p.ldd % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % (4 * sizeof(T)) == 0;
    const int warps = GRAD_THREADS / 32;
    const size_t smem = static_cast<size_t>(warps) * ((p.experts + 3) & ~3) * 4;
    const int grid = std::min((p.tokens + warps - 1) / warps, 8 * sm_count);
    const cudaError_t e = vec ? kernel_ready<route_grad_kernel<T, 4>>(0) : kernel_ready<route_grad_kernel<T, 1>>(0);
    if (e != cudaSuccess) return e;
    return vec ? launch_pdl(route_grad_kernel<T, 4>, grid, GRAD_THREADS, smem, a.stream, 1, p)
               : launch_pdl(route_grad_kernel<T, 1>, grid, GRAD_THREADS, smem, a.stream, 1, p);
}

}  // namespace

int route_chunks(int64_t tokens, int sm_count)
{
    if (tokens <= 64) return 1;
    return static_cast<int>(std::min<int64_t>((tokens + 31) / 32, sm_count));
}

size_t route_workspace(int64_t tokens, int64_t experts, int sm_count)
{
    const int chunks = route_chunks(tokens, sm_count);
    return chunks == 1 ? 0 : static_cast<size_t>(chunks) * (experts + 1) * 4;
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
    return a.bf16 ? launch_for<__nv_bfloat16>(p, a.stream, launches) : launch_for<float>(p, a.stream, launches);
}

cudaError_t launch_route_grad(const RouteGradArgs &a, int sm_count)
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
    return a.bf16 ? launch_grad<__nv_bfloat16>(a, p, sm_count) : launch_grad<float>(a, p, sm_count);
}

}  // namespace dg
