// Microscaled 4-bit floating point: E2M1 elements with one E8M0 scale per 32
// elements along K.  With e = max(floor(log2(max|x|)) - 2, -127) over a block,
// the scale byte is e + 127 and an element is the E2M1 value nearest to
// x * 2^-e (ties to the even code, magnitudes past 6 to 6); both steps are
// exact but for that one rounding.  A block that holds an infinity or a NaN
// gets the scale byte 0xFF (NaN) and zero codes.
#include <algorithm>
#include <cuda_bf16.h>

#include <cstdint>

#include "ragged.h"

namespace dg {
namespace {

constexpr int THREADS = 256;

// Eight E2M1 codes, element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Scale byte of a block from the largest magnitude's bits (NaN > infinity >
// finite as integers).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 2^(127 - byte), the reciprocal of the scale; 0 for the NaN scale (codes 0).
__device__ __forceinline__ float inverse_scale(uint32_t byte)
{
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); the lowest is subnormal, 0xFF is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fffffffu) : byte == 0u ? __uint_as_float(1u << 22) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// 8 elements of a row; vec: 16-byte loads are allowed.
__device__ __forceinline__ void load8(const float *s, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(s));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(s) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldg(s + i) : 0.0f;
    }
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *s, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(s));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(s[i]) : 0.0f;
    }
}

// One warp takes SEGS segments of 256 elements of a row: all its 16-byte loads
// are issued before the first is used, so a full SM has 128 KB (BF16) on the
// way.  Chunk w of the launch is row w / chunks, chunk w % chunks of it.
constexpr int SEGS = 4;

struct Chunk {
    long long row;
    int k;  // first element
};

__device__ __forceinline__ Chunk chunk_of(long long w, int chunks)
{
    Chunk c;
    if (w < (1ll << 31)) {  // 32-bit division where it fits
        const uint32_t r = static_cast<uint32_t>(w) / static_cast<uint32_t>(chunks);
        c.row = r;
        c.k = static_cast<int>(static_cast<uint32_t>(w) - r * chunks) * (SEGS * 256);
    } else {
        c.row = w / chunks;
        c.k = static_cast<int>(w - c.row * chunks) * (SEGS * 256);
    }
    return c;
}

// Rows along K: four lanes share a block, eight elements each.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantise_rows_kernel(const T *src, long long ld, int rows_per, long long stride, long long total, int K,
                         int chunks, int vec, uint8_t *codes, long long ldq, uint8_t *scales, long long lds)
{
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    if (w >= total) return;
    const Chunk c = chunk_of(w, chunks);
    const int Kp = (K + 31) / 32 * 32;
    const T *s = src + c.row * ld;
    if (stride) s = src + (c.row / rows_per) * stride + (c.row % rows_per) * ld;
    float v[SEGS][8];
#pragma unroll
    for (int j = 0; j < SEGS; ++j) {
        const int k = c.k + j * 256 + lane * 8;
        load8(s + k, K - k, vec != 0, v[j]);
    }
    uint32_t byte[SEGS];
#pragma unroll
    for (int j = 0; j < SEGS; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        byte[j] = scale_byte(m);
        const float inv = inverse_scale(byte[j]);
        const int k = c.k + j * 256 + lane * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = byte[j] == 255u ? 0.0f : v[j][i] * inv;
        if (k < Kp) *reinterpret_cast<uint32_t *>(codes + c.row * ldq + k / 2) = pack_e2m1(v[j]);
    }
    // the chunk's scale bytes, one a lane: segment lane / 8, block lane % 8
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < SEGS; ++j) {
        const uint32_t t = __shfl_sync(0xffffffffu, byte[j], (lane & 7) * 4);
        if ((lane >> 3) == j) mine = t;
    }
    if (c.k + lane * 32 < Kp) scales[c.row * lds + c.k / 32 + lane] = static_cast<uint8_t>(mine);
}

// K along the source's rows: one thread per block, neighbouring threads on
// neighbouring columns, so every load is a coalesced row segment.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantise_cols_kernel(const T *src, long long ld, int rows_per, long long stride, long long rows, int K,
                         int blocks, uint8_t *codes, long long ldq, uint8_t *scales, long long lds)
{
    const long long total = rows * blocks;
    for (long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * THREADS) {
        // order: batch, block of K, row
        const long long per_batch = static_cast<long long>(rows_per) * blocks;
        const long long b = i / per_batch;
        const long long in = i - b * per_batch;
        const int kb = static_cast<int>(in / rows_per);
        const int r = static_cast<int>(in - static_cast<long long>(kb) * rows_per);
        const T *s = src + b * stride + static_cast<long long>(kb) * 32 * ld + r;
        float v[32];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            v[k] = kb * 32 + k < K ? to_f32(s[k * ld]) : 0.0f;
            m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
        }
        const uint32_t byte = scale_byte(m);
        const float inv = inverse_scale(byte);
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = byte == 255u ? 0.0f : v[8 * j + k] * inv;
            out[j] = pack_e2m1(x);
        }
        const long long row = b * rows_per + r;
        *reinterpret_cast<uint4 *>(codes + row * ldq + kb * 16) = make_uint4(out[0], out[1], out[2], out[3]);
        scales[row * lds + kb] = static_cast<uint8_t>(byte);
    }
}

__device__ __forceinline__ void store8(float *d, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        reinterpret_cast<float4 *>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) d[i] = v[i];
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *d, int n, bool vec, const float (&v)[8])
{
    __nv_bfloat162 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    if (vec && n >= 8) {
        *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(w);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i < n) d[2 * i] = w[i].x;
            if (2 * i + 1 < n) d[2 * i + 1] = w[i].y;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
    dequantise_kernel(const uint8_t *codes, long long ldq, const uint8_t *scales, long long lds, long long total, int K,
                      int chunks, int vec, T *dst, long long ldd)
{
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    if (w >= total) return;
    const Chunk ch = chunk_of(w, chunks);
    uint32_t c[SEGS], byte[SEGS];
#pragma unroll
    for (int j = 0; j < SEGS; ++j) {
        const int k = ch.k + j * 256 + lane * 8;
        c[j] = byte[j] = 0;
        if (k < K) {
            c[j] = __ldg(reinterpret_cast<const uint32_t *>(codes + ch.row * ldq + k / 2));
            byte[j] = __ldg(scales + ch.row * lds + k / 32);
        }
    }
#pragma unroll
    for (int j = 0; j < SEGS; ++j) {
        const int k = ch.k + j * 256 + lane * 8;
        if (k >= K) break;
        const float scale = scale_value(byte[j]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t q = (c[j] >> (4 * i)) & 15u;
            // E2M1 magnitude: 0, 0.5, then (2 + mantissa) * 2^(exponent - 2)
            const float mag = (q & 7u) < 2u ? 0.5f * static_cast<float>(q & 1u)
                                            : __uint_as_float((((q & 6u) << 22) | ((q & 1u) << 22)) + (126u << 23));
            v[i] = ((q & 8u) ? -mag : mag) * scale;
        }
        store8(dst + ch.row * ldd + k, K - k, vec != 0, v);
    }
}

// One warp per chunk; block counts pass 2^31 - 1 only for matrices beyond memory.
int64_t chunk_blocks(int64_t chunks) { return (chunks + THREADS / 32 - 1) / (THREADS / 32); }

template <typename T>
cudaError_t quantise(bool k_rows, int64_t batch, int64_t rows, int64_t K, const T *src, int64_t ld, int64_t stride,
                     uint8_t *codes, int64_t ldq, uint8_t *scales, int64_t lds, int sm_count, cudaStream_t stream)
{
    const int64_t all = batch * rows;
    if (k_rows) {
        const int blocks = static_cast<int>((K + 31) / 32);
        const int grid = static_cast<int>(std::min<int64_t>((all * blocks + THREADS - 1) / THREADS, int64_t{sm_count} * 8));
        quantise_cols_kernel<T><<<grid, THREADS, 0, stream>>>(src, ld, static_cast<int>(rows), stride, all,
                                                              static_cast<int>(K), blocks, codes, ldq, scales, lds);
        return cudaGetLastError();
    }
    const int chunks = static_cast<int>((K + SEGS * 256 - 1) / (SEGS * 256));
    const int64_t grid = chunk_blocks(all * chunks);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t align = 16 / static_cast<int64_t>(sizeof(T));
    const int vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && ld % align == 0 && stride % align == 0;
    quantise_rows_kernel<T><<<static_cast<unsigned>(grid), THREADS, 0, stream>>>(
        src, ld, static_cast<int>(rows), stride, all * chunks, static_cast<int>(K), chunks, vec, codes, ldq, scales,
        lds);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dequantise(int64_t rows, int64_t K, const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                       T *dst, int64_t ldd, cudaStream_t stream)
{
    const int chunks = static_cast<int>((K + SEGS * 256 - 1) / (SEGS * 256));
    const int64_t grid = chunk_blocks(rows * chunks);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const int vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0 && (ldd * sizeof(T)) % 16 == 0;
    dequantise_kernel<T><<<static_cast<unsigned>(grid), THREADS, 0, stream>>>(
        codes, ldq, scales, lds, rows * chunks, static_cast<int>(K), chunks, vec, dst, ldd);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_quantise(bool k_rows, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                                int64_t stride, bool src_bf16, uint8_t *codes, int64_t ldq, uint8_t *scales,
                                int64_t lds, int sm_count, cudaStream_t stream)
{
    if (src_bf16)
        return quantise(k_rows, batch, rows, K, static_cast<const __nv_bfloat16 *>(src), ld, stride, codes, ldq,
                        scales, lds, sm_count, stream);
    return quantise(k_rows, batch, rows, K, static_cast<const float *>(src), ld, stride, codes, ldq, scales, lds,
                    sm_count, stream);
}

cudaError_t launch_mx4_dequantise(int64_t rows, int64_t K, const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                                  int64_t lds, void *dst, int64_t ldd, bool dst_bf16, cudaStream_t stream)
{
    if (dst_bf16)
        return dequantise(rows, K, codes, ldq, scales, lds, static_cast<__nv_bfloat16 *>(dst), ldd, stream);
    return dequantise(rows, K, codes, ldq, scales, lds, static_cast<float *>(dst), ldd, stream);
}

}  // namespace dg
