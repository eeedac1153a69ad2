// 8-bit integers with one FP32 scale a row: s = max|x| / 127 rounded to FP32,
// codes x / s rounded to the nearest integer, ties to even, within -127 .. 127.
// The quotient is taken as if in infinite precision: it lies between x times a
// reciprocal of s rounded down and one rounded up, and where these two round to
// different integers (one element in 20000) the exact remainder x - c * s decides.  A row of zeros has scale
// 0; one that holds an infinity or a NaN has scale NaN; both have codes 0.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight elements of a row as they are loaded (vec: 16-byte loads are allowed;
// past the row's end zeros), and widened.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    // from shared memory, the second half `pitch` bytes behind (n elements are there)
    __device__ __forceinline__ void fetch(uint32_t from, int pitch, int n)
    {
        a = lds_f4(from);
        if (n > 4) b = lds_f4(from + pitch);
    }
    __device__ __forceinline__ void load(const float *s, int n, bool vec)
    {
        if (vec && n >= 8) {
            a = *reinterpret_cast<const float4 *>(s);
            b = *(reinterpret_cast<const float4 *>(s) + 1);
        } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? s[i] : 0.0f;
            a = make_float4(v[0], v[1], v[2], v[3]);
            b = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    // the largest magnitude's bits, and the most of two such
    __device__ __forceinline__ uint32_t top(uint32_t m) const
    {
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        return m;
    }
    static __device__ __forceinline__ uint32_t whole(uint32_t m) { return m; }
    __device__ __forceinline__ void widen(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void fetch(uint32_t from, int, int) { a = lds_u4(from); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *s, int n, bool vec)
    {
        if (vec && n >= 8) {
            a = *reinterpret_cast<const uint4 *>(s);
        } else {
            const uint16_t *t = reinterpret_cast<const uint16_t *>(s);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (2 * i < n ? uint32_t{t[2 * i]} : 0u) | (2 * i + 1 < n ? uint32_t{t[2 * i + 1]} << 16 : 0u);
            a = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // as above, of the even and the odd elements in the halves of a word
    __device__ __forceinline__ uint32_t top(uint32_t m) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return m;
    }
    static __device__ __forceinline__ uint32_t whole(uint32_t m) { return max(m & 0xffff0000u, m << 16); }
    __device__ __forceinline__ void widen(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// The scale of a row from the largest magnitude's bits (NaN > infinity > finite
// as integers).
__device__ __forceinline__ float scale_of(uint32_t amax_bits)
{
    return amax_bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
}

// Codes of values by a row's scale.
struct Coder {
    float scale, low, high;  // reciprocals, 2^-22 below and above
    bool none, small;
    __device__ __forceinline__ explicit Coder(float s) : scale(s)
    {
        none = !(s > 0.0f);
        small = s < 1e-30f;  // no FP32 reciprocal to rely on
        const float inverse = none || small ? 0.0f : 1.0f / s;
        low = inverse * (1.0f - 0x1p-22f);
        high = inverse * (1.0f + 0x1p-22f);
    }
    // Where the rounding is open.  The remainder is exact: a multiple of half a
    // unit of the scale's last place, and little more than half the scale.
    __device__ __forceinline__ int settle(float x) const
    {
        if (small) return static_cast<int>(fmin(fmax(rint(static_cast<double>(x) / scale), -127.0), 127.0));
        float c = rintf(x * low);
        const float d = fmaf(-c, scale, x), twice = 2.0f * fabsf(d);
        if (twice > scale || (twice == scale && (static_cast<int>(c) & 1))) c += copysignf(1.0f, d);
        return static_cast<int>(c);
    }
    // Eight codes.  Adding 1.5 * 2^23 rounds to an integer and leaves it in the
    // low bits; |x| <= 127 s keeps it within -127 .. 127.
    __device__ __forceinline__ uint2 operator()(const float (&v)[8]) const
    {
        if (none) return make_uint2(0u, 0u);
        constexpr float ROUND = 12582912.0f;
        const auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
        };
        const auto codes = [&](float r) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(fmaf(v[i], r, ROUND));
            return make_uint2(four(w[0], w[1], w[2], w[3]), four(w[4], w[5], w[6], w[7]));
        };
        const uint2 a = codes(low), b = codes(high);
        if (a.x == b.x && a.y == b.y && !small) return a;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = static_cast<uint32_t>(settle(v[i]));
        return make_uint2(four(w[0], w[1], w[2], w[3]), four(w[4], w[5], w[6], w[7]));
    }
};

__device__ __forceinline__ void store8(int8_t *dst, uint2 c, int n)
{
    if (n >= 8) {
        *reinterpret_cast<uint2 *>(dst) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) dst[i] = static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

__host__ __device__ constexpr int quantise_threads(int tpr) { return tpr > THREADS ? tpr : THREADS; }

// TPR threads a row, U pieces of eight elements a thread (U = 0: any number, and
// the row is read again for the codes).  Few pieces a thread: eight left so few
// warps that 8192 x 14336 took 270 us.  S > 0 (rows on 16-byte boundaries): a
// thread's pieces of the next S - 1 rows are on their way into shared memory while
// it works on one, each thread's own, so that no barrier comes into it.  The issue
// of instructions is 74 % used then, memory 36 to 43 % (8192 x 4096 and 12001 x 4096
// BF16: 25 and 34 us).
template <typename T, int TPR, int U, int S>
__global__ void __launch_bounds__(quantise_threads(TPR))
    quantise_kernel(const T *src, long long ld, long long stride, long long rows, long long all, int K, bool vec,
                    int8_t *codes, long long ldq, float *scales)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint32_t part[32];
    constexpr int NT = quantise_threads(TPR), ROWS = NT / TPR, WORDS = sizeof(Raw<T>) / 16, RING = S > 0 ? S : 1;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int pieces = (K + 7) / 8;
    const long long step = static_cast<long long>(gridDim.x) * ROWS;
    griddep_wait();
    griddep_launch_dependents();
    const auto row_at = [&](long long r) {
        const long long b = r / rows;
        return src + b * stride + (r - b * rows) * ld;
    };
    const uint32_t mine = S > 0 ? smem_addr(ring) + threadIdx.x * 16 : 0u;
    const auto slot = [&](int s, int u, int w) { return mine + static_cast<uint32_t>(((s * U + u) * WORDS + w) * NT * 16); };
    const auto request = [&](long long r, int s) {
        if (r < all) {
            const T *row = row_at(r);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    constexpr int N = 16 / sizeof(T);
                    const int k = (u * TPR + t) * 8 + w * N, left = (K - k) * static_cast<int>(sizeof(T));
                    if (left > 0) cp_async_16(slot(s, u, w), row + k, left < 16 ? static_cast<uint32_t>(left) : 16u);
                }
        }
        cp_async_commit();
    };
    if (S > 0) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s) request(static_cast<long long>(blockIdx.x) * ROWS + sub + s * step, s);
    }
    int stage = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * ROWS; r0 < all; r0 += step) {
        const long long r = r0 + sub;
        const bool there = r < all;
        const T *row = there ? row_at(r) : src;
        Raw<T> kept[U > 0 ? U : 1];
        uint32_t amax = 0;
        if (S > 0) {
            request(r + (S - 1) * step, (stage + S - 1) % RING);
            cp_async_wait<S - 1>();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                kept[u].clear();
                if (there && (u * TPR + t) * 8 < K) kept[u].fetch(slot(stage, u, 0), NT * 16, K - (u * TPR + t) * 8);
                amax = kept[u].top(amax);
            }
            stage = (stage + 1) % RING;
        } else if (U > 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (u * TPR + t) * 8;
                kept[u].load(row + k, there ? K - k : 0, vec);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) amax = kept[u].top(amax);
        } else if (there) {
            for (int i = t; i < pieces; i += TPR) {
                kept[0].load(row + i * 8, K - i * 8, vec);
                amax = kept[0].top(amax);
            }
        }
        amax = __reduce_max_sync(0xffffffffu, Raw<T>::whole(amax));
        if (TPR > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) amax = max(amax, part[sub * (TPR / 32) + w]);
            __syncthreads();  // part is written again for the next row
        }
        const Coder q(scale_of(amax));
        if (there && t == 0) scales[r] = q.scale;
        int8_t *out = codes + r * ldq;
        const auto put = [&](const Raw<T> &raw, int k) {
            float v[8];
            raw.widen(v);
            store8(out + k, q(v), K - k);
        };
        if (U > 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (u * TPR + t) * 8;
                if (there && k < K) put(kept[u], k);
            }
        } else if (there) {
            for (int i = t; i < pieces; i += TPR) {
                kept[0].load(row + i * 8, K - i * 8, vec);
                put(kept[0], i * 8);
            }
        }
    }
}

// Row-major weights: element (r, k) at src[k * ld + r].  A CTA takes 32 rows of
// the output at a time: the maxima of its 32 columns, then 128 values of K at a
// time through shared memory.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantise_turn_kernel(const T *src, long long ld, long long stride, int rows, long long all, int K, int8_t *codes,
                         long long ldq, float *scales)
{
    constexpr int W = THREADS / 32;
    __shared__ uint32_t part[W][32];
    __shared__ __align__(16) int8_t tile[32][128 + 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch_dependents();
    const int blocks = (rows + 31) / 32;  // of a matrix
    const int out_row = threadIdx.x >> 3, piece = (threadIdx.x & 7) * 16;
    for (long long u = blockIdx.x; u < all; u += gridDim.x) {
        const long long b = u / blocks;
        const int r0 = static_cast<int>(u - b * blocks) * 32, r = r0 + lane;
        const T *col = src + b * stride + r;
        uint32_t amax = 0;
        if (r < rows)
#pragma unroll 8
            for (int k = warp; k < K; k += W)
                amax = max(amax, __float_as_uint(to_f32(col[static_cast<long long>(k) * ld])) & 0x7fffffffu);
        part[warp][lane] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) amax = max(amax, part[w][lane]);
        const Coder q(scale_of(amax));
        const long long first = b * rows + r0;
        if (warp == 0 && r < rows) scales[first + lane] = q.scale;
        for (int k0 = 0; k0 < K; k0 += 128) {
#pragma unroll
            for (int j = warp * 8; j < 128; j += W * 8) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = r < rows && k0 + j + i < K ? to_f32(col[static_cast<long long>(k0 + j + i) * ld]) : 0.0f;
                *reinterpret_cast<uint2 *>(&tile[lane][j]) = q(v);
            }
            __syncthreads();
            if (r0 + out_row < rows) {
                int8_t *dst = codes + (first + out_row) * ldq + k0 + piece;
                const int n = K - k0 - piece;
                const uint4 v = *reinterpret_cast<const uint4 *>(&tile[out_row][piece]);
                if (n >= 16) {
                    *reinterpret_cast<uint4 *>(dst) = v;
                } else {
                    store8(dst, make_uint2(v.x, v.y), n);
                    store8(dst + 8, make_uint2(v.z, v.w), n - 8);
                }
            }
            __syncthreads();  // tile, and after the last part, is written again
        }
    }
}

__device__ __forceinline__ void put8(float *dst, const float (&v)[8], int n, bool vec)
{
    if (vec && n >= 8) {
        *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *(reinterpret_cast<float4 *>(dst) + 1) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) dst[i] = v[i];
    }
}

__device__ __forceinline__ void put8(__nv_bfloat16 *dst, const float (&v)[8], int n, bool vec)
{
    if (vec && n >= 8) {
        const __nv_bfloat162 w[4] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3]),
                                     __floats2bfloat162_rn(v[4], v[5]), __floats2bfloat162_rn(v[6], v[7])};
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) dst[i] = __float2bfloat16_rn(v[i]);
    }
}

// A warp takes 256 elements of a row.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    dequantise_kernel(long long rows, int K, const int8_t *codes, long long ldq, const float *scales, T *dst,
                      long long ldd, bool vec)
{
    griddep_wait();
    griddep_launch_dependents();
    const int chunks = (K + 255) / 256, lane = threadIdx.x & 31;
    const long long all = rows * chunks;
    for (long long w = blockIdx.x * (THREADS / 32LL) + (threadIdx.x >> 5); w < all; w += gridDim.x * (THREADS / 32LL)) {
        const long long r = w / chunks;
        const int k = static_cast<int>(w - r * chunks) * 256 + lane * 8, n = K - k;
        if (n <= 0) continue;
        const float s = scales[r];
        float v[8];
        if (n >= 8) {
            const uint2 c = *reinterpret_cast<const uint2 *>(codes + r * ldq + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)))) * s;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? static_cast<float>(codes[r * ldq + k + i]) * s : 0.0f;
        }
        put8(dst + r * ldd + k, v, n, vec);
    }
}

// A warp takes WIDEN x 512 codes of a row, 16 a lane at a time.  Rows are read
// up to the end of their last 16 bytes, which the pitch holds, and written so.
constexpr int WIDEN = 4;

__global__ void __launch_bounds__(THREADS)
    widen_kernel(const int8_t *src, long long ld, long long rows, int K, __half *dst)
{
    griddep_wait();
    griddep_launch_dependents();
    const int pieces = (K + 15) / 16, chunks = (pieces + 32 * WIDEN - 1) / (32 * WIDEN), lane = threadIdx.x & 31;
    const long long pitch = pieces * 16LL, all = rows * chunks;
    for (long long w = blockIdx.x * (THREADS / 32LL) + (threadIdx.x >> 5); w < all; w += gridDim.x * (THREADS / 32LL)) {
        const long long row = w / chunks;
        const int p0 = static_cast<int>(w - row * chunks) * 32 * WIDEN + lane;
        const uint4 *from = reinterpret_cast<const uint4 *>(src + row * ld);
        uint4 *to = reinterpret_cast<uint4 *>(dst + row * pitch);
        uint4 c[WIDEN];
#pragma unroll
        for (int i = 0; i < WIDEN; ++i)
            if (p0 + i * 32 < pieces) c[i] = from[p0 + i * 32];
#pragma unroll
        for (int i = 0; i < WIDEN; ++i)
            if (p0 + i * 32 < pieces) {
                uint4 lo, hi;
                i8_to_f16(c[i], lo, hi);
                to[2 * (p0 + i * 32)] = lo;
                to[2 * (p0 + i * 32) + 1] = hi;
            }
    }
}

int grid_for(long long units, int per_cta, int per_sm, int sm_count, int max_ctas)
{
    return capped(std::max(1LL, std::min<long long>((units + per_cta - 1) / per_cta, int64_t{per_sm} * sm_count)), max_ctas);
}

template <typename T, int TPR, int U, int S>
cudaError_t launch_quantise_form(const void *src, int64_t ld, int64_t stride, int64_t batch, int64_t rows, int64_t K,
                                 bool vec, int8_t *codes, int64_t ldq, float *scales, int sm_count, int max_ctas,
                                 cudaStream_t stream)
{
    constexpr int NT = quantise_threads(TPR);
    constexpr size_t SMEM = static_cast<size_t>(S) * U * NT * sizeof(Raw<T>);
    const cudaError_t e = kernel_ready<quantise_kernel<T, TPR, U, S>>(SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(quantise_kernel<T, TPR, U, S>, grid_for(batch * rows, NT / TPR, 2048 / NT, sm_count, max_ctas), NT, SMEM,
                      stream, 1, static_cast<const T *>(src), static_cast<long long>(ld),
                      static_cast<long long>(stride), static_cast<long long>(rows),
                      static_cast<long long>(batch * rows), static_cast<int>(K), vec, codes,
                      static_cast<long long>(ldq), scales);
}

template <typename T, int TPR, int U>
cudaError_t launch_quantise(const void *src, int64_t ld, int64_t stride, int64_t batch, int64_t rows, int64_t K,
                            int8_t *codes, int64_t ldq, float *scales, int sm_count, int max_ctas,
                            cudaStream_t stream)
{
    const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && (ld * sizeof(T)) % 16 == 0 &&
                     (stride * sizeof(T)) % 16 == 0;
    // more rows than run at once: those that follow are fetched ahead
    constexpr int S = sizeof(T) == 2 ? 4 : 3;
    if (U > 0 && vec && batch * rows > static_cast<int64_t>(quantise_threads(TPR) / TPR) * 2 * sm_count)
        return launch_quantise_form<T, TPR, U, U == 0 ? 0 : S>(src, ld, stride, batch, rows, K, vec, codes, ldq, scales,
                                                               sm_count, max_ctas, stream);
    return launch_quantise_form<T, TPR, U, 0>(src, ld, stride, batch, rows, K, vec, codes, ldq, scales, sm_count,
                                              max_ctas, stream);
}

template <typename T>
cudaError_t launch_quantise_for(bool k_rows, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                                int64_t stride, int8_t *codes, int64_t ldq, float *scales, int sm_count, int max_ctas,
                                cudaStream_t stream)
{
    if (k_rows) {
        const int64_t all = batch * ((rows + 31) / 32);
        const cudaError_t e = kernel_ready<quantise_turn_kernel<T>>(0);
        if (e != cudaSuccess) return e;
        return launch_pdl(quantise_turn_kernel<T>, capped(all, max_ctas), THREADS, 0, stream, 1,
                          static_cast<const T *>(src), static_cast<long long>(ld), static_cast<long long>(stride),
                          static_cast<int>(rows), static_cast<long long>(all), static_cast<int>(K), codes,
                          static_cast<long long>(ldq), scales);
    }
    const auto run = [&](auto f) {
        return f(src, ld, stride, batch, rows, K, codes, ldq, scales, sm_count, max_ctas, stream);
    };
    if (K <= 256) return run(launch_quantise<T, 32, 1>);
    if (K <= 1024) return run(launch_quantise<T, 32, 4>);
    if (K <= 2048) return run(launch_quantise<T, 256, 1>);
    if (K <= 4096) return run(launch_quantise<T, 256, 2>);
    if (K <= 8192) return run(launch_quantise<T, 512, 2>);
    if (K <= 16384) return run(launch_quantise<T, 1024, 2>);
    return run(launch_quantise<T, 1024, 0>);
}

}  // namespace

cudaError_t launch_i8_quantise(bool k_rows, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                               int64_t stride, bool src_bf16, int8_t *codes, int64_t ldq, float *scales, int sm_count,
                               int max_ctas, cudaStream_t stream)
{
    return src_bf16 ? launch_quantise_for<__nv_bfloat16>(k_rows, batch, rows, K, src, ld, stride, codes, ldq, scales,
                                                         sm_count, max_ctas, stream)
                    : launch_quantise_for<float>(k_rows, batch, rows, K, src, ld, stride, codes, ldq, scales, sm_count,
                                                 max_ctas, stream);
}

cudaError_t launch_i8_dequantise(int64_t rows, int64_t K, const int8_t *codes, int64_t ldq, const float *scales,
                                 void *dst, int64_t ldd, bool dst_bf16, int sm_count, int max_ctas,
                                 cudaStream_t stream)
{
    const int es = dst_bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0 && (ldd * es) % 16 == 0;
    const int grid = grid_for(rows * ((K + 255) / 256), THREADS / 32, 8, sm_count, max_ctas);
    cudaError_t e;
    if (dst_bf16) {
        e = kernel_ready<dequantise_kernel<__nv_bfloat16>>(0);
        return e != cudaSuccess ? e
                                : launch_pdl(dequantise_kernel<__nv_bfloat16>, grid, THREADS, 0, stream, 1,
                                             static_cast<long long>(rows), static_cast<int>(K), codes,
                                             static_cast<long long>(ldq), scales, static_cast<__nv_bfloat16 *>(dst),
                                             static_cast<long long>(ldd), vec);
    }
    e = kernel_ready<dequantise_kernel<float>>(0);
    return e != cudaSuccess ? e
                            : launch_pdl(dequantise_kernel<float>, grid, THREADS, 0, stream, 1,
                                         static_cast<long long>(rows), static_cast<int>(K), codes,
                                         static_cast<long long>(ldq), scales, static_cast<float *>(dst),
                                         static_cast<long long>(ldd), vec);
}

cudaError_t launch_i8_widen(const int8_t *src, int64_t ld, int64_t rows, int64_t K, void *dst, int sm_count,
                            int max_ctas, cudaStream_t stream)
{
    const int64_t chunks = (K + 512 * WIDEN - 1) / (512 * WIDEN);
    const cudaError_t e = kernel_ready<widen_kernel>(0);
    if (e != cudaSuccess) return e;
    return launch_pdl(widen_kernel, grid_for(rows * chunks, THREADS / 32, 8, sm_count, max_ctas), THREADS, 0, stream, 1, src,
                      static_cast<long long>(ld), static_cast<long long>(rows), static_cast<int>(K),
                      static_cast<__half *>(dst));
}

}  // namespace dg
