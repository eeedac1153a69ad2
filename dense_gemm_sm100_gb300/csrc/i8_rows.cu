// 8-bit products of few rows: C[r][n] = (sum_k a(r, k) b(n, k)) sa[r] sb[n] for
// groups of a few rows each, as decoding has them.  Reading B once is all that
// counts there, and the tensor-core kernel's hand-overs (bytes, FP16 in tensor
// memory, product) take longer than a tile's bytes.
//
// A pass takes up to MR rows of one group; the units of work are CH neighbouring
// rows of B in a pass, shared out evenly over the CTAs, so that a group of many rows
// (all 256 rows in one of 128 groups of 768 x 2048, in the L2 cache: 16 us) is spread
// as well as many groups of one (37 us).  More passes over a group read B out of the
// L2 cache, four rows of A at a time: that is the worst case, see kFewRowsOfGroup.
//
// A warp takes a unit at a time, 16 bytes of each row a lane and step; AHEAD loads
// of a lane, two to four steps, are under way while it works on one, across the
// units' ends (started anew for every unit, 14336 x 4096 took 17 us; 14.5 us now,
// 4.0 TB/s).  The rows of A lie in shared memory, MR of them, and four-way integer
// dot products add into 32-bit integers, exact up to K = 131071 (shared memory holds
// up to K = 24576 for MR = 4).  In the end the
// CH x MR = 16 sums of all lanes are added in a butterfly that halves their number
// at every step.  With MR = 8 the dot products and the reads of A, twice as many
// for every byte of B, set the pace (17 us).
#include <algorithm>
#include <cuda_bf16.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int SUMS = 16;   // of a warp: rows of B times rows of A
constexpr int A_BYTES = 96 * 1024, MAX_PASSES = 1536;  // two CTAs fit an SM
constexpr int AHEAD = 8;   // 16-byte loads of a lane under way

struct RowsParams {
    const long long *offsets;  // null: one group of all rows
    int groups, rows, N, K, pieces, kpad;  // 16-byte pieces of K, K in whole rounds of steps
    const int8_t *a, *b;
    long long lda, ldb;
    const float *sa, *sb;
    void *C;
    long long ldc;
    int *status;
};

__device__ __forceinline__ void put(float *c, float v) { *c = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *c, float v) { *c = __float2bfloat16_rn(v); }

// Threads over groups: for every MR rows of a group (at most) its number and the
// first of them, in order, and how many such there are.  Offsets that do not rise
// within [0, rows] are reported, and there are none then.
template <int MR>
__device__ int passes_of(const RowsParams &p, int2 *list, int *sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.offsets == nullptr) {
        const int all = (p.rows + MR - 1) / MR;
        for (int i = tid; i < all; i += THREADS) list[i] = make_int2(0, i * MR);
        __syncthreads();
        return all;
    }
    const int per = (p.groups + THREADS - 1) / THREADS;
    const int g0 = min(p.groups, tid * per), g1 = min(p.groups, g0 + per);
    int n = 0, bad = 0;
    for (int g = g0; g < g1; ++g) {
        const long long lo = p.offsets[g], hi = p.offsets[g + 1];
        if (lo < 0 || hi < lo || hi > p.rows)
            bad = 1;
        else
            n += (static_cast<int>(hi - lo) + MR - 1) / MR;
    }
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 31) sums[warp] = inc;
    bad = __syncthreads_or(bad);
    if (bad) {
        if (blockIdx.x == 0 && tid == 0) atomicCAS(p.status, 0, kStatusBadOffsets);
        return 0;
    }
    int at = inc - n, all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += sums[w];
        all += sums[w];
    }
    for (int g = g0; g < g1; ++g) {
        const int m = static_cast<int>(p.offsets[g + 1] - p.offsets[g]);
        for (int r = 0; r < m; r += MR) list[at++] = make_int2(g, r);
    }
    __syncthreads();
    return all;
}

template <int MR, typename T>
__global__ void __launch_bounds__(THREADS, 2) rows_kernel(const RowsParams p)
{
    constexpr int CH = SUMS / MR;    // rows of B of a warp
    constexpr int BUFS = AHEAD / CH;  // steps under way
    extern __shared__ __align__(16) uint8_t smem[];  // A's rows, then the list of passes
    __shared__ int sums[WARPS];
    int2 *list = reinterpret_cast<int2 *>(smem + static_cast<size_t>(MR) * p.kpad);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (p.N + CH - 1) / CH, steps = p.kpad / 512;  // a multiple of BUFS
    // B's rows of this CTA's first units towards the L2 cache while the kernel before
    // this one (the quantisation of A) still runs: a hint, whatever B holds by then.
    if (p.offsets == nullptr) {
        const int lines = (p.pieces + 7) / 8;
        const long long first = static_cast<long long>(blocks) * blockIdx.x / gridDim.x * CH;
        for (int i = tid; i < WARPS * CH * lines; i += THREADS) {
            const long long n = first + i / lines;
            if (n < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.b + n * p.ldb + i % lines * 128));
        }
    }
    griddep_wait();
    const long long units = static_cast<long long>(passes_of<MR>(p, list, sums)) * blocks;
    const uint32_t a_base = smem_addr(smem);
    // A run of neighbouring units a CTA, pass by pass.
    const long long end = units * (blockIdx.x + 1LL) / gridDim.x;
    for (long long u = units * blockIdx.x / gridDim.x; u < end;) {
        const int which = static_cast<int>(u / blocks), g = list[which].x, r0 = list[which].y;
        const int q0 = static_cast<int>(u - static_cast<long long>(which) * blocks);
        const int q1 = static_cast<int>(min(static_cast<long long>(blocks), q0 + (end - u)));
        const long long lo = p.offsets ? p.offsets[g] : 0, hi = p.offsets ? p.offsets[g + 1] : p.rows;
        const int m = static_cast<int>(hi - lo);
        const int8_t *base = p.b + static_cast<long long>(g) * p.N * p.ldb;
        // the loads that run ahead: step `fs` of unit `fq`
        int fq = q0 + warp, fs = 0;
        const uint4 *from[CH];
        const auto rows_of = [&](int q) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                from[j] = reinterpret_cast<const uint4 *>(base + static_cast<long long>(min(q * CH + j, p.N - 1)) * p.ldb);
        };
        uint4 buf[BUFS][CH];
        const auto fetch = [&](uint4(&w)[CH]) {
            const int c = fs * 32 + lane;
            if (fq < q1 && c < p.pieces)
#pragma unroll
                for (int j = 0; j < CH; ++j) w[j] = __ldg(from[j] + c);
            if (++fs == steps) {
                fs = 0;
                fq += WARPS;
                if (fq < q1) rows_of(fq);
            }
        };
        if (fq < q1) rows_of(fq);
#pragma unroll
        for (int x = 0; x < BUFS; ++x) {
#pragma unroll
            for (int j = 0; j < CH; ++j) buf[x][j] = make_uint4(0u, 0u, 0u, 0u);
            fetch(buf[x]);
        }
        __syncthreads();  // nobody reads the rows of A before
        const int quads = p.kpad / 16;
        for (int i = tid; i < MR * quads; i += THREADS) {
            const int r = i / quads, c = i - r * quads, left = p.K - c * 16;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + r < m && left > 0) {
                v = *reinterpret_cast<const uint4 *>(p.a + (lo + r0 + r) * p.lda + c * 16);
                if (left < 16) {  // zeros past K, where B may hold anything
                    const auto keep = [&](uint32_t w, int n) {
                        return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
                    };
                    v = make_uint4(keep(v.x, left), keep(v.y, left - 4), keep(v.z, left - 8), keep(v.w, left - 12));
                }
            }
            sts_u4(a_base + i * 16, v);
        }
        __syncthreads();
        for (int q = q0 + warp; q < q1; q += WARPS) {
            int acc[SUMS];
#pragma unroll
            for (int i = 0; i < SUMS; ++i) acc[i] = 0;
#pragma unroll 1
            for (int s = 0; s < steps; s += BUFS) {
#pragma unroll
                for (int x = 0; x < BUFS; ++x) {
                    uint4 w[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) w[j] = buf[x][j];
                    fetch(buf[x]);
                    const uint32_t at = a_base + ((s + x) * 32 + lane) * 16;
#pragma unroll
                    for (int r = 0; r < MR; ++r) {
                        const uint4 a = lds_u4(at + r * p.kpad);
#pragma unroll
                        for (int j = 0; j < CH; ++j) {
                            int t = acc[j * MR + r];
                            t = __dp4a(static_cast<int>(a.x), static_cast<int>(w[j].x), t);
                            t = __dp4a(static_cast<int>(a.y), static_cast<int>(w[j].y), t);
                            t = __dp4a(static_cast<int>(a.z), static_cast<int>(w[j].z), t);
                            acc[j * MR + r] = __dp4a(static_cast<int>(a.w), static_cast<int>(w[j].w), t);
                        }
                    }
                }
            }
            // the sums of all lanes: the upper half of the values goes to the
            // lanes that have the bit set, the lower half to the others
#pragma unroll
            for (int d = 16; d >= 2; d >>= 1) {
                const bool up = (lane & d) != 0;
                const int half = d / 2;
#pragma unroll
                for (int i = 0; i < SUMS / 2; ++i)
                    if (i < half) {
                        const int send = up ? acc[i] : acc[i + half], stay = up ? acc[i + half] : acc[i];
                        acc[i] = stay + __shfl_xor_sync(0xffffffffu, send, d);
                    }
            }
            const int sum = acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
            const int value = lane >> 1, n = q * CH + value / MR, r = r0 + value % MR;
            if ((lane & 1) == 0 && n < p.N && r < m) {
                const float v = static_cast<float>(sum) * p.sa[lo + r] * p.sb[static_cast<long long>(g) * p.N + n];
                put(static_cast<T *>(p.C) + (lo + r) * p.ldc + n, v);
            }
        }
        u += q1 - q0;
    }
}

// K in whole rounds of the steps under way.
int64_t padded(int64_t K, int mr)
{
    const int64_t round = 512 * AHEAD / (SUMS / mr);
    return (K + round - 1) / round * round;
}

template <int MR, typename T>
cudaError_t launch(const RowsParams &p, int sm_count, int max_ctas, cudaStream_t stream)
{
    constexpr size_t MOST = A_BYTES + MAX_PASSES * sizeof(int2);
    const cudaError_t e = kernel_ready<rows_kernel<MR, T>>(MOST);
    if (e != cudaSuccess) return e;
    constexpr int CH = SUMS / MR;
    const long long units = static_cast<long long>(p.rows) * ((p.N + CH - 1) / CH);  // at most
    const int grid = capped(std::min<long long>((units + WARPS - 1) / WARPS, 2LL * sm_count), max_ctas);
    const size_t smem = static_cast<size_t>(MR) * p.kpad + static_cast<size_t>(p.rows) * sizeof(int2);
    return launch_pdl(rows_kernel<MR, T>, grid, THREADS, smem, stream, 1, p);
}

}  // namespace

bool i8_rows_fit(int64_t rows, int64_t K, int mr)
{
    return K > 0 && mr * padded(K, mr) <= A_BYTES && rows <= MAX_PASSES;
}

cudaError_t launch_i8_rows(const RaggedArgs &r, int mr, const int8_t *a, int64_t lda, const int8_t *b, int64_t ldb,
                           int sm_count, int max_ctas)
{
    RowsParams p;
    p.offsets = reinterpret_cast<const long long *>(r.offsets);
    p.groups = r.groups;
    p.rows = r.rows;
    p.N = r.P;
    p.K = r.K;
    p.pieces = (r.K + 15) / 16;
    p.kpad = static_cast<int>(padded(r.K, mr));
    p.a = a;
    p.b = b;
    p.lda = lda;
    p.ldb = ldb;
    p.sa = r.row_scale_q;
    p.sb = r.row_scale_p;
    p.C = r.C;
    p.ldc = r.ldc;
    p.status = r.status;
    if (mr == 4)
        return r.out_bf16 ? launch<4, __nv_bfloat16>(p, sm_count, max_ctas, r.stream)
                          : launch<4, float>(p, sm_count, max_ctas, r.stream);
    return r.out_bf16 ? launch<8, __nv_bfloat16>(p, sm_count, max_ctas, r.stream)
                      : launch<8, float>(p, sm_count, max_ctas, r.stream);
}

}  // namespace dg
