// Microscaled 4-bit floating point: E2M1 elements with one E8M0 scale per 32
// elements along K.  With e = max(floor(log2(max|x|)) - 2, -127) over a block,
// the scale byte is e + 127 and an element is the E2M1 value nearest to
// x * 2^-e (ties to the even code, magnitudes past 6 to 6); both steps are
// exact but for that one rounding.  A block that holds an infinity or a NaN
// gets the scale byte 0xFF (NaN) and zero codes.
#include <algorithm>
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
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

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x)
{
    return static_cast<T>(x);
}

// 8 elements of a row as they are loaded (vec: 16-byte loads are allowed), and
// widened.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
};

__device__ __forceinline__ void load8(const float *s, int n, bool vec, Raw<float> &r)
{
    if (vec && n >= 8) {
        r.a = *reinterpret_cast<const float4 *>(s);
        r.b = *(reinterpret_cast<const float4 *>(s) + 1);
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? *(s + i) : 0.0f;
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *s, int n, bool vec, Raw<__nv_bfloat16> &r)
{
    if (vec && n >= 8) {
        r.a = *reinterpret_cast<const uint4 *>(s);
    } else {
        const uint16_t *t = reinterpret_cast<const uint16_t *>(s);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (2 * i < n ? uint32_t{*(t + 2 * i)} : 0u) | (2 * i + 1 < n ? uint32_t{*(t + 2 * i + 1)} << 16 : 0u);
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ void widen(const Raw<float> &r, float (&v)[8])
{
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
    v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}

__device__ __forceinline__ void widen(const Raw<__nv_bfloat16> &r, float (&v)[8])
{
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Memory sets the time: 16384 x 8192 BF16 quantised in 55 us (6.1 TB/s of
// reads and writes) and turned back in 58 us (5.8).  A warp takes chunks of
// SEGS segments of 256 elements of a row, 64 bytes a lane, and issues the loads
// of its next chunk before it works on the present one, so loads are on the way
// all the time (without: 88 us).
template <typename T>
constexpr int kSegs = sizeof(T) == 2 ? 4 : 2;

// Position of a warp in the rows x chunks grid, advanced by a fixed step
// without division.
struct Cursor {
    long long row, step_row;
    int chunk, step_chunk, chunks;
    __device__ Cursor(long long first, long long step, int n) : chunks(n)
    {
        row = first / n;
        chunk = static_cast<int>(first - row * n);
        step_row = step / n;
        step_chunk = static_cast<int>(step - step_row * n);
    }
    __device__ void next()
    {
        row += step_row;
        chunk += step_chunk;
        if (chunk >= chunks) {
            chunk -= chunks;
            ++row;
        }
    }
};

// Rows along K: four lanes share a block, eight elements each.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantise_rows_kernel(const T *src, long long ld, int rows_per, long long stride, long long rows, int K,
                         int chunks, int vec, uint8_t *codes, long long ldq, uint8_t *scales, long long lds)
{
    constexpr int SEGS = kSegs<T>;
    griddep_wait();
    const int lane = threadIdx.x & 31;
    Cursor at(static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5),
              static_cast<long long>(gridDim.x) * (THREADS / 32), chunks);
    const int Kp = (K + 31) / 32 * 32;
    Raw<T> next[SEGS];
    const auto fetch = [&]() {
        if (at.row >= rows) return;
        const T *s = stride ? src + (at.row / rows_per) * stride + (at.row % rows_per) * ld : src + at.row * ld;
#pragma unroll
        for (int j = 0; j < SEGS; ++j) {
            const int k = (at.chunk * SEGS + j) * 256 + lane * 8;
            load8(s + k, K - k, vec != 0, next[j]);
        }
    };
    fetch();
    while (at.row < rows) {
        float v[SEGS][8];
#pragma unroll
        for (int j = 0; j < SEGS; ++j) widen(next[j], v[j]);
        const long long row = at.row;
        const int k0 = at.chunk * (SEGS * 256);
        at.next();
        fetch();
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
            const int k = k0 + j * 256 + lane * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] *= inv;
            if (k < Kp)
                *reinterpret_cast<uint32_t *>(codes + row * ldq + k / 2) = byte[j] == 255u ? 0u : pack_e2m1(v[j]);
        }
        // the chunk's scale bytes, one a lane: segment lane / 8, block lane % 8
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < SEGS; ++j) {
            const uint32_t t = __shfl_sync(0xffffffffu, byte[j], (lane & 7) * 4);
            if ((lane >> 3) == j) mine = t;
        }
        if (lane < SEGS * 8 && k0 + lane * 32 < Kp) scales[row * lds + k0 / 32 + lane] = static_cast<uint8_t>(mine);
    }
    griddep_launch_dependents();
}

// K along the source's rows.  A CTA turns tiles of COLS source columns (output
// rows) by 256 elements of K: a thread takes two blocks of one column, so that
// every load is part of a coalesced row segment; codes and scales meet in
// shared memory and leave as 128 and 8 contiguous bytes of an output row.
// 4096 x 14336 BF16 in 34 us, 4.4 TB/s; 72 us when the loads of a block were
// guarded one by one, which kept the compiler from issuing them together.
constexpr int COLS = 64;
constexpr int COL_PITCH = 144;  // bytes of a row's codes in shared memory: 16-byte stores without conflicts

template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantise_cols_kernel(const T *src, long long ld, int rows_per, long long stride, int batch, int K, int blocks,
                         uint8_t *codes, long long ldq, uint8_t *scales, long long lds)
{
    __shared__ __align__(16) uint8_t s_codes[COLS * COL_PITCH];
    __shared__ __align__(8) uint8_t s_scales[COLS * 8];
    const int tid = threadIdx.x;
    const int c = tid % COLS, g = tid / COLS;  // column; first block
    const int tiles_r = (rows_per + COLS - 1) / COLS, tiles_k = (blocks + 7) / 8;
    const long long total = static_cast<long long>(batch) * tiles_r * tiles_k;
    griddep_wait();
    for (long long i = blockIdx.x; i < total; i += gridDim.x) {
        const long long bk = i / tiles_r;  // order: matrix, tile of K, tile of columns
        const int r0 = static_cast<int>(i - bk * tiles_r) * COLS;
        const long long b = bk / tiles_k;
        const int kb0 = static_cast<int>(bk - b * tiles_k) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kb = kb0 + g + 4 * h;
            const T *s = src + b * stride + static_cast<long long>(kb) * 32 * ld + r0 + c;
            const int n = r0 + c < rows_per ? K - kb * 32 : 0;  // elements of the block
            T raw[32];  // all loads before the first use
            if (n >= 32) {
#pragma unroll
                for (int k = 0; k < 32; ++k) raw[k] = s[k * ld];
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) raw[k] = k < n ? s[k * ld] : from_f32<T>(0.0f);
            }
            float v[32];
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                v[k] = to_f32(raw[k]);
                m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
            }
            const uint32_t byte = scale_byte(m);
            const float inv = inverse_scale(byte);
            uint32_t out[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = v[8 * j + k] * inv;
                out[j] = byte == 255u ? 0u : pack_e2m1(x);
            }
            *reinterpret_cast<uint4 *>(s_codes + c * COL_PITCH + (g + 4 * h) * 16) =
                make_uint4(out[0], out[1], out[2], out[3]);
            s_scales[c * 8 + g + 4 * h] = static_cast<uint8_t>(byte);
        }
        __syncthreads();
        const long long row0 = b * rows_per + r0;
        const int left = blocks - kb0;  // blocks of the tile
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 32 + (tid >> 3), piece = tid & 7;
            if (r0 + r < rows_per && piece < left)
                *reinterpret_cast<uint4 *>(codes + (row0 + r) * ldq + (kb0 + piece) * 16) =
                    *reinterpret_cast<const uint4 *>(s_codes + r * COL_PITCH + piece * 16);
        }
        if (tid < COLS && r0 + tid < rows_per) {
            uint8_t *d = scales + (row0 + tid) * lds + kb0;
            if (left >= 8) {
                *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<const uint2 *>(s_scales + tid * 8);
            } else {
                for (int j = 0; j < left; ++j) d[j] = s_scales[tid * 8 + j];
            }
        }
        __syncthreads();
    }
    griddep_launch_dependents();
}

// A scale twice, as BF16: the lowest is subnormal, 0xFF is NaN.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t byte)
{
    return (byte == 255u ? 0x7fffu : byte == 0u ? 0x0040u : byte << 7) * 0x00010001u;
}

// Codes as BF16 pairs.  A code's bits s, e e, m placed at the sign, the
// two lowest exponent bits and the highest mantissa bit of a BF16 number are
// its value times 2^-126 (the codes 0 and 0.5 as a zero and a subnormal), so
// two exact multiplications, by 2^126 and by the scale, give the element.
template <int PAIRS>
__device__ __forceinline__ void expand(uint32_t c, __nv_bfloat162 scale, __nv_bfloat162 (&w)[PAIRS])
{
    const uint32_t even = c & 0x0f0f0f0fu, odd = (c >> 4) & 0x0f0f0f0fu;
    const uint32_t up = 0x7e807e80u;  // 2^126 twice
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        // byte i of `even` in the low half, of `odd` in the high half
        const uint32_t t = __byte_perm(even, odd, 0x0400u + 0x1111u * i);
        const uint32_t bits = ((t << 6) & 0x01c001c0u) | ((t << 12) & 0x80008000u);
        w[i] = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&bits),
                               *reinterpret_cast<const __nv_bfloat162 *>(&up)),
                       scale);
    }
}

__device__ __forceinline__ void store8(float *d, int n, bool vec, const __nv_bfloat162 (&w)[4])
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __low2float(w[i]);
        v[2 * i + 1] = __high2float(w[i]);
    }
    if (vec && n >= 8) {
        reinterpret_cast<float4 *>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) d[i] = v[i];
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *d, int n, bool vec, const __nv_bfloat162 (&w)[4])
{
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
    dequantise_kernel(const uint8_t *codes, long long ldq, const uint8_t *scales, long long lds, long long rows, int K,
                      int chunks, int vec, T *dst, long long ldd)
{
    constexpr int SEGS = kSegs<T>;
    griddep_wait();
    const int lane = threadIdx.x & 31;
    Cursor at(static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5),
              static_cast<long long>(gridDim.x) * (THREADS / 32), chunks);
    uint32_t c[SEGS], byte[SEGS];
    const auto fetch = [&]() {
        if (at.row >= rows) return;
#pragma unroll
        for (int j = 0; j < SEGS; ++j) {
            const int k = (at.chunk * SEGS + j) * 256 + lane * 8;
            if (k < K) {
                c[j] = *reinterpret_cast<const uint32_t *>(codes + at.row * ldq + k / 2);
                byte[j] = *(scales + at.row * lds + k / 32);
            }
        }
    };
    fetch();
    while (at.row < rows) {
        uint32_t code[SEGS], s[SEGS];
#pragma unroll
        for (int j = 0; j < SEGS; ++j) code[j] = c[j], s[j] = byte[j];
        T *d = dst + at.row * ldd;
        const int k0 = at.chunk * (SEGS * 256);
        at.next();
        fetch();
        if (sizeof(T) == 4 && vec != 0) {
            // FP32: four elements a lane and store, 512 contiguous bytes a warp;
            // their codes are half a word of lane 16 h + lane / 2 (137 us for
            // 16384 x 8192 with eight elements a lane, 32 bytes apart)
#pragma unroll
            for (int j = 0; j < 2 * SEGS; ++j) {
                const int from = (j & 1) * 16 + (lane >> 1);
                const uint32_t c4 = __shfl_sync(0xffffffffu, code[j >> 1], from) >> ((lane & 1) * 16);
                const uint32_t both = scale_bf16x2(__shfl_sync(0xffffffffu, s[j >> 1], from));
                const int k = k0 + j * 128 + lane * 4;
                if (k >= K) continue;
                __nv_bfloat162 w[2];
                expand<2>(c4 & 0xffffu, *reinterpret_cast<const __nv_bfloat162 *>(&both), w);
                const float4 v = make_float4(__low2float(w[0]), __high2float(w[0]), __low2float(w[1]), __high2float(w[1]));
                float *f = reinterpret_cast<float *>(d) + k;
                if (k + 4 <= K) {
                    *reinterpret_cast<float4 *>(f) = v;
                } else {
                    f[0] = v.x;
                    if (k + 1 < K) f[1] = v.y;
                    if (k + 2 < K) f[2] = v.z;
                }
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < SEGS; ++j) {
            const int k = k0 + j * 256 + lane * 8;
            if (k >= K) break;
            const uint32_t both = scale_bf16x2(s[j]);
            __nv_bfloat162 w[4];
            expand<4>(code[j], *reinterpret_cast<const __nv_bfloat162 *>(&both), w);
            store8(d + k, K - k, vec != 0, w);
        }
    }
    griddep_launch_dependents();
}

// Launches that may start while the kernel before them on the stream ends
// (each kernel waits for it before its first access to memory): a product
// behind the quantisation of its operand then finds its set-up done.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Blocks of eight warps, one chunk a warp at least, eight blocks an SM at most.
int chunk_grid(int64_t chunks, int sm_count)
{
    const int64_t blocks = (chunks + THREADS / 32 - 1) / (THREADS / 32);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t{sm_count} * 8)));
}

template <typename T>
cudaError_t quantise(bool k_rows, int64_t batch, int64_t rows, int64_t K, const T *src, int64_t ld, int64_t stride,
                     uint8_t *codes, int64_t ldq, uint8_t *scales, int64_t lds, int sm_count, cudaStream_t stream)
{
    const int64_t all = batch * rows;
    if (k_rows) {
        const int blocks = static_cast<int>((K + 31) / 32);
        const int64_t tiles = batch * ((rows + COLS - 1) / COLS) * ((blocks + 7) / 8);
        const int grid = static_cast<int>(std::min<int64_t>(tiles, int64_t{sm_count} * 8));
        return launch(quantise_cols_kernel<T>, grid, stream, src, ld, rows, stride, batch, K, blocks, codes, ldq,
                      scales, lds);
    }
    const int chunks = static_cast<int>((K + kSegs<T> * 256 - 1) / (kSegs<T> * 256));
    const int64_t align = 16 / static_cast<int64_t>(sizeof(T));
    const int vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && ld % align == 0 && stride % align == 0;
    return launch(quantise_rows_kernel<T>, chunk_grid(all * chunks, sm_count), stream, src, ld, rows, stride, all, K,
                  chunks, vec, codes, ldq, scales, lds);
}

template <typename T>
cudaError_t dequantise(int64_t rows, int64_t K, const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                       T *dst, int64_t ldd, int sm_count, cudaStream_t stream)
{
    const int chunks = static_cast<int>((K + kSegs<T> * 256 - 1) / (kSegs<T> * 256));
    const int vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0 && (ldd * sizeof(T)) % 16 == 0;
    return launch(dequantise_kernel<T>, chunk_grid(rows * chunks, sm_count), stream, codes, ldq, scales, lds, rows, K,
                  chunks, vec, dst, ldd);
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
                                  int64_t lds, void *dst, int64_t ldd, bool dst_bf16, int sm_count,
                                  cudaStream_t stream)
{
    if (dst_bf16)
        return dequantise(rows, K, codes, ldq, scales, lds, static_cast<__nv_bfloat16 *>(dst), ldd, sm_count, stream);
    return dequantise(rows, K, codes, ldq, scales, lds, static_cast<float *>(dst), ldd, sm_count, stream);
}

}  // namespace dg
