// Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T, on the tensor cores.
//
// Three products a step, each with its epilogue: A = X X^T; B = b A + c A A;
// X' = a X + B X.  A and B are symmetric: only tiles on and below the diagonal
// are computed, and what lies below is written twice.
//
// Numbers.  The products' operands are FP16 (11 bits; BF16's 8 would cost a
// relative 1e-2 to 4e-2 of the result), scaled by powers of two so that FP16's
// range fits: X by 2^12, A by 2^11, B by 2^10.  A step multiplies what is small
// in X by a = 3.4, five steps by 485, so it matters where roundings fall
// (simulated in FP64, of the result's norm, gradients with a few strong
// directions and noise / plain noise): all operands rounded to FP16 3.5e-3 /
// 1.3e-3; the term a X taken from X in two FP16 numbers, its rest beside the
// value, 3e-4 / 1.5e-3; the diagonals of A and B, their largest elements, kept
// out of the products and applied in FP32 in the epilogues as well 2.7e-4 /
// 7e-4; BF16's rounding of the result is 1.7e-3.  With E the part of A off the
// diagonal and d the diagonal, A A = E E + (d_i + d_j) E + d^2.  FP32 results
// take both FP16 numbers of every operand: three products (the fourth is below
// 2^-22 of the first), and sums cut into segments that are added to nearest.
//
// The norm.  X is stored as Y = G 2^e with the norm of Y in [2^12, 2^13): exact
// for BF16 and FP32 alike, the rest of 1 / (|G| + eps) enters A's and X's first
// epilogues.  X is Y 2^-q, q = 12 where |G| outweighs eps.  Where eps outweighs
// |G|, X is tiny and q larger, and as long as A is too small to hold it back X
// grows by a = 3.4 or more a step: every X epilogue takes out of Y, and of q, the
// whole powers of two by which a bound on Y's norm has grown past 2^14, until q is
// 12.  Each matrix has its own q and bound, in turn in two places, so that a launch
// writes what the next one reads.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "ortho.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr int BP = 128;               // rows of P one CTA stages
constexpr int BK = 64;                // K elements of a ring stage
constexpr int P_BYTES = BP * 128;
constexpr int MAX_STAGES = 12;
constexpr int TMEM_COLS = 512;
constexpr int ACC1 = 256;             // the second accumulator's column
constexpr int NUM_BARS = 2 * MAX_STAGES + 2 + 2 + 1;
constexpr int EPI_WARPS = 8;
constexpr int EPI_BYTES = EPI_WARPS * 4096;  // a warp's 32 x 32 values
constexpr int WARPS = 2 + EPI_WARPS;
constexpr int THREADS = 32 * WARPS;
constexpr int SMEM_MAX = 227 * 1024;
constexpr int SEG = 4;                // ring stages of a segment of a two-term sum
constexpr float SCALE_A = 2048.0f, SCALE_B = 1024.0f;
constexpr int SCALE_X_LOG = 12;

// factors of a matrix, see below; the last two twice, by X's buffer that is read
enum Factor : int { kFactorRest = 0, kFactorUp0, kFactorUp1, kFactorLog, kFactorMost = kFactorLog + 2 };
constexpr int FACTORS = ORTHO_FACTORS;

struct Params {
    int m, n, ldm, ldn, batch;
    int bn, tiles_i, tiles, stages, stage_bytes, q_bytes, kt;
    int first, last, has_rest, from;
    float ca, cb, cc;
    const __half *x[2];  // planes of X as read
    __half *x_out[2];
    __half *a[2], *b[2];
    float *da, *db;
    float *factors;
    void *o;
    long long ldo, stride_o;
    int turned, o_bf16, o_vec;
    int *status;
    unsigned long long timeout_ns;
    int debug_drop;
};

struct Tile {
    int b, i0, j0;  // matrix, first row (of the CTA pair), first column
    bool mirror;    // wholly below the diagonal
    bool some;      // it has columns
};

// Symmetric products (r = rows of a tile / its columns): block row I holds the
// r (I + 1) tiles up to the diagonal; block columns past m are empty.
template <int CG, bool SYM>
__device__ __forceinline__ Tile tile_at(const Params &p, int u)
{
    constexpr int BM = CG * BP;
    Tile t;
    t.b = u / p.tiles;
    const int k = u - t.b * p.tiles;
    int I, J;
    if (SYM) {
        const int r = max(1, BM / p.bn);
        I = static_cast<int>((sqrtf(8.0f * static_cast<float>(k) / static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while (r * (I * (I + 1) / 2) > k) --I;
        while (r * ((I + 1) * (I + 2) / 2) <= k) ++I;
        J = k - r * (I * (I + 1) / 2);
        t.mirror = J / r < I;
    } else {
        J = k / p.tiles_i;
        I = k - J * p.tiles_i;
        t.mirror = false;
    }
    t.i0 = I * BM;
    t.j0 = J * p.bn;
    t.some = t.j0 < (SYM ? p.m : p.n);
    return t;
}

// 2^-k for k >= 0; 0 past FP32's normal numbers.
__device__ __forceinline__ float power_down(int k) { return __int_as_float(max(0, 127 - k) << 23); }

// Eight FP16 numbers added to v.
__device__ __forceinline__ void add8(uint4 w, float (&v)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
        v[2 * i] += f.x;
        v[2 * i + 1] += f.y;
    }
}

// Eight values in FP16, and what that leaves of them.
__device__ __forceinline__ uint4 round8(const float (&v)[8], float (&rest)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(h);
        rest[2 * i] = v[2 * i] - f.x;
        rest[2 * i + 1] = v[2 * i + 1] - f.y;
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 round8(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// SPLIT: operands of two FP16 numbers.  STEP: X' = a X + B X, Q = X with its
// rows as K; else A or B, symmetric, P and Q the same matrix along K.
// UNITS: 16-column units of a tile that a warp adds up (SPLIT; 8 for tiles of more
// than 128 columns, whose sums take 128 registers a thread and leave some spilled);
// 2 for tiles of 32 columns (X: 64).  What the epilogue adds is loaded right before it is
// added where sums are held: loaded a chunk ahead, it spilled (13 FP32 matrices of
// 1020 x 520 466 -> 516 us replayed).
template <int CG, bool SPLIT, int STEP, int UNITS>
__global__ void __launch_bounds__(THREADS, 1)
    ortho_kernel(const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmP1,
                 const __grid_constant__ CUtensorMap tmQ0, const __grid_constant__ CUtensorMap tmQ1, const Params p)
{
    constexpr int PLANES = SPLIT ? 2 : 1;
    constexpr bool XSTEP = STEP == kOrthoX;
    // FP16 operands, FP32 accumulator; Q MN-major for X
    constexpr uint32_t IDESC = (1u << 4) | ((XSTEP ? 1u : 0u) << 16) | (static_cast<uint32_t>((CG * BP) >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
    const uint32_t sbase = raw_addr + pad;
    const uint32_t epi_base = sbase + static_cast<uint32_t>(p.stages * p.stage_bytes);
    const uint32_t bars = epi_base + EPI_BYTES;
    const uint32_t full_bar = bars;                         // [stages], used in the even CTA
    const uint32_t empty_bar = full_bar + 8 * MAX_STAGES;   // [stages]
    const uint32_t tfull_bar = empty_bar + 8 * MAX_STAGES;  // [2]
    const uint32_t tempty_bar = tfull_bar + 16;             // [2], used in the even CTA
    const uint32_t drain_bar = tempty_bar + 16;
    uint8_t *tail = smem_raw + pad + p.stages * p.stage_bytes + EPI_BYTES + NUM_BARS * 8;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int first_unit = blockIdx.x / CG, unit_step = gridDim.x / CG;
    const int num_units = p.tiles * p.batch;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar + 8 * b, 1);
            mbar_init(tempty_bar + 8 * b, EPI_WARPS * CG);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmP0);
        tma_prefetch_desc(&tmQ0);
    }
    if (warp == 1) {
        const uint32_t slot = smem_addr(const_cast<uint32_t *>(tmem_slot));
        if (CG == 2) {
            tmem_alloc_pair(slot, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(slot, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    if (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            const int q_cta = p.bn / CG;
            const uint32_t tx = static_cast<uint32_t>(CG * PLANES * (P_BYTES + p.q_bytes));
            uint32_t it = 0, s = 0, ph = 0;
            bool ok = true;
            for (int u = first_unit; ok && u < num_units; u += unit_step) {
                const Tile t = tile_at<CG, !XSTEP>(p, u);
                if (!t.some) continue;
                const int pi = t.i0 + static_cast<int>(rank) * BP;
                const int qj = t.j0 + static_cast<int>(rank) * q_cta;
                for (int kt = 0; kt < p.kt; ++kt, ++it) {
                    if (!mbar_wait(empty_bar + 8 * s, ph ^ 1u, abort_flag, p.status, kWaitProducerEmpty,
                                   p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = full_bar + 8 * s;
                    const uint32_t fb = CG == 2 ? mapa_shared(fb_local, 0) : fb_local;
                    const uint32_t st = sbase + s * p.stage_bytes;
                    if (leader) mbar_arrive_expect_tx(fb_local, tx);
                    if (++s == static_cast<uint32_t>(p.stages)) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (p.debug_drop && blockIdx.x == 0 && it == 0) continue;  // bytes that never come
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl) {
                        const CUtensorMap *mp = pl ? &tmP1 : &tmP0, *mq = pl ? &tmQ1 : &tmQ0;
                        const uint32_t p_st = st + pl * P_BYTES, q_st = st + PLANES * P_BYTES + pl * p.q_bytes;
                        if (CG == 2)
                            tma_load_3d_pair(p_st, mp, fb, kt * BK, pi, t.b);
                        else
                            tma_load_3d(p_st, mp, fb, kt * BK, pi, t.b);
                        if (XSTEP) {  // chunks of 64 columns by 64 rows of K
                            if (CG == 2)
                                tma_load_4d_pair(q_st, mq, fb, 0, kt * BK, qj / 64, t.b);
                            else
                                tma_load_4d(q_st, mq, fb, 0, kt * BK, qj / 64, t.b);
                        } else {
                            if (CG == 2)
                                tma_load_3d_pair(q_st, mq, fb, kt * BK, qj, t.b);
                            else
                                tma_load_3d(q_st, mq, fb, kt * BK, qj, t.b);
                        }
                    }
                }
            }
            // Stages issued last, oldest first: (s, ph) is the next one.
            const uint32_t n = min(it, static_cast<uint32_t>(p.stages));
            uint32_t ds = s >= n ? s - n : s + p.stages - n;
            uint32_t dph = s >= n ? ph : ph ^ 1u;
            for (uint32_t i = 0; i < n; ++i) {
                int dummy = 0;
                if (ok) {
                    // every release must have landed before shared memory goes away
                    mbar_wait(empty_bar + 8 * ds, dph, abort_flag, p.status, kWaitDrain, p.timeout_ns);
                } else if (leader) {
                    // after an abort: leave no copy in flight
                    mbar_wait(full_bar + 8 * ds, dph, &dummy, nullptr, kWaitDrain, p.timeout_ns);
                }
                if (++ds == static_cast<uint32_t>(p.stages)) {
                    ds = 0;
                    dph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer (even CTA)
        if (leader) {
            const uint32_t idesc = IDESC | (static_cast<uint32_t>(p.bn >> 3) << 17);
            uint32_t s = 0, ph = 0, acc_it = 0;
            bool ok = true, issued = false;
            for (int u = first_unit; ok && u < num_units; u += unit_step) {
                if (!tile_at<CG, !XSTEP>(p, u).some) continue;
                for (int seg0 = 0; seg0 < p.kt; seg0 += SPLIT ? SEG : p.kt, ++acc_it) {
                    const int seg1 = SPLIT ? min(p.kt, seg0 + SEG) : p.kt;
                    const uint32_t abuf = acc_it & 1u;
                    if (!mbar_wait_warp(tempty_bar + 8 * abuf, ((acc_it >> 1) & 1u) ^ 1u, abort_flag, p.status,
                                        kWaitMmaTmemEmpty, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + abuf * ACC1;
                    for (int kt = seg0; kt < seg1; ++kt) {
                        if (!mbar_wait_warp(full_bar + 8 * s, ph, abort_flag, p.status, kWaitMmaFull, p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t p_st = sbase + s * p.stage_bytes, q_st = p_st + PLANES * P_BYTES;
                        if (elect_one()) {
                            // value x value, then value x rest and rest x value
#pragma unroll
                            for (int term = 0; term < (SPLIT ? 3 : 1); ++term) {
                                const uint32_t pa = p_st + (term == 2 ? P_BYTES : 0);
                                const uint32_t qa = q_st + (term == 1 ? p.q_bytes : 0);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    const uint64_t pd = smem_desc(pa + kk * 32, 16, 1024, kLayoutSw128);
                                    const uint64_t qd = XSTEP ? smem_desc(qa + kk * 16 * 128, BK * 128, 1024, kLayoutSw128)
                                                              : smem_desc(qa + kk * 32, 16, 1024, kLayoutSw128);
                                    const uint32_t acc = kt > seg0 || kk > 0 || term > 0 ? 1u : 0u;
                                    if (CG == 2)
                                        tc_mma_f16_pair(d_tmem, pd, qd, idesc, acc);
                                    else
                                        tc_mma_f16(d_tmem, pd, qd, idesc, acc);
                                }
                            }
                            if (CG == 2)
                                tc_commit_pair_multicast(empty_bar + 8 * s, 0x3);
                            else
                                tc_commit(empty_bar + 8 * s);
                        }
                        __syncwarp();
                        issued = true;
                        if (++s == static_cast<uint32_t>(p.stages)) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (elect_one()) {
                        if (CG == 2)
                            tc_commit_pair_multicast(tfull_bar + 8 * abuf, 0x3);
                        else
                            tc_commit(tfull_bar + 8 * abuf);
                    }
                    __syncwarp();
                }
            }
            if (!ok && issued && lane == 0) {
                // Let every MMA already issued finish before TMEM is freed.
                if (CG == 2)
                    tc_commit_pair_multicast(drain_bar, 0x1);
                else
                    tc_commit(drain_bar);
                int dummy = 0;
                mbar_wait(drain_bar, 0, &dummy, nullptr, kWaitDrain, p.timeout_ns);
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        // A warp turns 32 x 32 sums in shared memory so that a lane holds 8
        // neighbouring columns of rows lane / 4, + 8, + 16, + 24: loads and stores
        // of 16 bytes a lane touch 8 lines an instruction.  (With a row a lane
        // they touched 32, and the line look-ups set the pace: X of 16 matrices of
        // 4096 x 2048 500 us, B 150 us.)
        const int q = warp & 3;            // tensor-memory lane quarter
        const int half = (warp - 2) >> 2;  // 0: even chunks of 32 columns, 1: odd ones
        // Tiles of 32 columns: both halves take the one chunk, 16 of its rows each (with
        // half of the warps idle one matrix of 256 x 384 took 83.7 us, 80.3 now; in the
        // kernel of the other tiles the choice cost 3 % of 16 matrices of 4096 x 2048).
        constexpr bool narrow = UNITS == 2 && !XSTEP;
        const int mine = UNITS == 2 ? 1 : (p.bn / 32 + 1 - half) / 2;
        const uint32_t stage = epi_base + static_cast<uint32_t>(warp - 2) * 4096;
        const int sub = lane >> 2, piece = lane & 3;
        // 16 bytes c of row r: bank conflicts are spread over the rows
        const auto at = [&](int r, int c) { return stage + r * 128 + ((c ^ (r & 7)) * 16); };
        uint32_t acc_it = 0;
        bool ok = true;
        for (int u = first_unit; ok && u < num_units; u += unit_step) {
            const Tile t = tile_at<CG, !XSTEP>(p, u);
            if (!t.some) continue;
            const int i0 = t.i0 + static_cast<int>(rank) * BP + q * 32;  // the warp's first row
            const long long mat = t.b;
            float *f = p.factors + mat * FACTORS;
            const int log_x = static_cast<int>(f[kFactorLog + p.from]);  // X = Y 2^-log_x
            const float rest = p.first ? f[kFactorRest] : 1.0f;
            // With the powers of two of what is read and written in the constants, a
            // value is acc * scale (A), + e * (row + column) (B; e an element of A,
            // row and column from the diagonal), or + x * row (X).
            float scale, row_c[4], row_d[4], column_c = 0.0f;  // rows i0 + sub, + 8, ...
            if (XSTEP) {
                int take = 0;  // powers of two taken out of Y
                float most = 0.0f;
                if (log_x > SCALE_X_LOG) {
                    most = f[kFactorMost + p.from];
                    const float s = most * power_down(log_x), s2 = s * s;  // no singular value of X is larger
                    most *= fabsf(p.ca) + s2 * (fabsf(p.cb) + s2 * fabsf(p.cc));
                    const int log_most = (__float_as_int(most) >> 23) - 127;  // rounded down
                    take = max(0, min(log_x - SCALE_X_LOG, log_most - SCALE_X_LOG - 1));
                }
                if (!p.last && i0 == 0 && t.j0 == 0 && half == 0 && lane == 0) {
                    f[kFactorLog + (p.from ^ 1)] = static_cast<float>(log_x - take);
                    f[kFactorMost + (p.from ^ 1)] = most * power_down(take);
                }
                // a result may lie below FP32's normal numbers
                const float post = rest * (p.last ? ldexpf(1.0f, -log_x) : power_down(take));
                scale = post / SCALE_B;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i0 + sub + 8 * r;
                    row_c[r] = i < p.m ? (p.ca + p.db[mat * p.ldm + i]) * post : 0.0f;
                }
            } else if (STEP == kOrthoA) {
                scale = rest * rest * power_down(2 * log_x) * SCALE_A;
            } else {
                scale = p.cc * (SCALE_B / (SCALE_A * SCALE_A));
                column_c = p.cc * (SCALE_B / SCALE_A);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i0 + sub + 8 * r;
                    row_d[r] = i < p.m ? p.da[mat * p.ldm + i] : 0.0f;
                    row_c[r] = fmaf(p.cc, row_d[r], p.cb) * (SCALE_B / SCALE_A);
                }
            }
            const int width = XSTEP ? p.n : p.m, ld = XSTEP ? p.ldn : p.ldm;
            const long long rows = mat * p.m;

            const auto await = [&]() {
                const uint32_t abuf = acc_it & 1u;
                ok = mbar_wait_warp(tfull_bar + 8 * abuf, (acc_it >> 1) & 1u, abort_flag, p.status, kWaitEpiTmemFull,
                                    p.timeout_ns);
                tc_fence_after_sync();
                return ok;
            };
            const auto release = [&]() {  // relaxed: see ragged.cu
                const uint32_t bar = tempty_bar + 8 * (acc_it & 1u);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive_relaxed(bar);
                    else
                        mbar_arrive_cluster_relaxed(mapa_shared(bar, 0));
                }
                ++acc_it;
            };
            const auto load = [&](int unit, uint32_t(&v)[16]) {
                tmem_load_16cols(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc_it & 1u) * ACC1 + unit * 16, v);
            };
            // Chunk k of this warp: columns from column(k) on.
            const auto column = [&](int k) { return narrow ? t.j0 : t.j0 + (2 * k + half) * 32; };
            const auto skips = [&](int r) { return narrow && (r >> 1) != half; };
            const auto turn = [&](const uint32_t(&lo)[16], const uint32_t(&hi)[16]) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sts_u4(at(lane, c), make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]));
                    sts_u4(at(lane, c + 4), make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]));
                }
                __syncwarp();
            };
            // The operands that the epilogue adds: X, or A where B is made.
            uint4 extra[2][4];
            float4 diagonal[2];  // A's, at a lane's columns (narrow: loaded ahead)
            const bool reads = XSTEP || STEP == kOrthoB;
            const bool two = SPLIT || (XSTEP && p.has_rest);
            const auto load_diagonal = [&](int j) {
                const float4 *d = reinterpret_cast<const float4 *>(p.da + mat * p.ldm + j);
                diagonal[0] = d[0];
                diagonal[1] = d[1];
            };
            const auto fetch = [&](int k) {
                if (!reads) return;
                const int j = column(k) + piece * 8;
                const __half *const *from = XSTEP ? p.x : p.a;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (skips(r)) continue;
                    const int i = i0 + sub + 8 * r;
                    const bool in = i < p.m && j < width;
                    const long long o = (rows + i) * ld + j;
                    extra[0][r] = in ? *reinterpret_cast<const uint4 *>(from[0] + o) : make_uint4(0u, 0u, 0u, 0u);
                    if (two) extra[1][r] = in ? *reinterpret_cast<const uint4 *>(from[1] + o) : make_uint4(0u, 0u, 0u, 0u);
                }
                if (narrow && j < width) load_diagonal(j);
            };
            const bool back = XSTEP ? p.last && p.turned : t.mirror;  // results are needed column by column
            __half *const *planes = XSTEP ? p.x_out : STEP == kOrthoA ? p.a : p.b;
            const auto finish = [&](int k) {
                const int jc = column(k), j = jc + piece * 8;
                if (jc >= width) {
                    __syncwarp();
                    return;
                }
                float dj[8];
                if (!XSTEP && STEP == kOrthoB && j < width) {
                    if (!narrow) load_diagonal(j);
                    const float4 d0 = diagonal[0], d1 = diagonal[1];
                    dj[0] = d0.x, dj[1] = d0.y, dj[2] = d0.z, dj[3] = d0.w;
                    dj[4] = d1.x, dj[5] = d1.y, dj[6] = d1.z, dj[7] = d1.w;
#pragma unroll
                    for (int c = 0; c < 8; ++c) dj[c] *= column_c;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = sub + 8 * r, i = i0 + row;
                    if (i >= p.m || j >= width || skips(r)) continue;
                    const float4 a0 = lds_f4(at(row, 2 * piece)), a1 = lds_f4(at(row, 2 * piece + 1));
                    float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w}, e[8] = {};
                    if (reads) {
                        add8(extra[0][r], e);
                        if (two) add8(extra[1][r], e);
                    }
                    if (!XSTEP && i >= j && i < j + 8) {
                        // the diagonal, kept in FP32 and out of the matrix
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (j + c == i) {
                                if (STEP == kOrthoA) {
                                    p.da[mat * p.ldm + i] = v[c] * scale * (1.0f / SCALE_A);
                                } else {
                                    const float d = narrow ? row_d[r] : p.da[mat * p.ldm + i];
                                    p.db[mat * p.ldm + i] =
                                        p.cb * d + p.cc * fmaf(d, d, v[c] * (1.0f / (SCALE_A * SCALE_A)));
                                }
                                v[c] = e[c] = 0.0f;
                            }
                    }
                    const float rc = reads ? row_c[r] : 0.0f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        v[c] *= scale;
                        if (XSTEP)
                            v[c] = fmaf(e[c], rc, v[c]);
                        else if (STEP == kOrthoB)
                            v[c] = fmaf(e[c], rc + dj[c], v[c]);
                    }
                    const long long o = (rows + i) * ld + j;
                    if (!XSTEP || !p.last) {
                        if (SPLIT || XSTEP) {
                            float rest[8];
                            *reinterpret_cast<uint4 *>(planes[0] + o) = round8(v, rest);
                            *reinterpret_cast<uint4 *>(planes[1] + o) = round8(rest);
                        } else {
                            *reinterpret_cast<uint4 *>(planes[0] + o) = round8(v);
                        }
                    } else if (!p.turned) {
                        const long long to = mat * p.stride_o + i * p.ldo + j;
                        if (p.o_bf16) {
                            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.o) + to;
                            if (p.o_vec && j + 8 <= p.n) {
                                uint32_t y[4];
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
                                    y[c] = *reinterpret_cast<const uint32_t *>(&b);
                                }
                                *reinterpret_cast<uint4 *>(out) = make_uint4(y[0], y[1], y[2], y[3]);
                            } else {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    if (j + c < p.n) out[c] = __float2bfloat16_rn(v[c]);
                            }
                        } else {
                            float *out = static_cast<float *>(p.o) + to;
                            if (p.o_vec && j + 8 <= p.n) {
                                *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
                                *(reinterpret_cast<float4 *>(out) + 1) = make_float4(v[4], v[5], v[6], v[7]);
                            } else {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    if (j + c < p.n) out[c] = v[c];
                            }
                        }
                    }
                    if (back) {
                        sts_f4(at(row, 2 * piece), make_float4(v[0], v[1], v[2], v[3]));
                        sts_f4(at(row, 2 * piece + 1), make_float4(v[4], v[5], v[6], v[7]));
                    }
                }
                __syncwarp();
                if (!back) return;
                if constexpr (narrow) {
                    // as below, 8 pairs of rows and 4 columns an instruction
                    const int r = half * 16 + (lane & 7) * 2, h = lane >> 3;
                    const uint32_t base = stage + r * 128 + h * 4;
                    __half *to = planes[0] + (rows + jc + h) * p.ldm + i0 + r;
                    const long long step = 4LL * p.ldm, left = i0 + r < p.m ? p.m - jc - h : 0,
                                    rest = SPLIT ? planes[1] - planes[0] : 0;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const uint32_t c = n ^ (r & 7);
                        const float v0 = lds_f1(base + c * 16), v1 = lds_f1(base + 128 + (c ^ 1) * 16);
                        if (4 * n < left) {
                            const __half2 b = __floats2half2_rn(v0, v1);
                            *reinterpret_cast<__half2 *>(to) = b;
                            if (SPLIT) {
                                const float2 w = __half22float2(b);
                                *reinterpret_cast<__half2 *>(to + rest) = __floats2half2_rn(v0 - w.x, v1 - w.y);
                            }
                        }
                        to += step;
                    }
                } else if (!XSTEP) {
                    // Column c of the result is row jc + c of the mirrored half: rows r and
                    // r + 1 of the tile a lane, columns 2 n and 2 n + 1 an instruction.
                    const int r = (lane & 15) * 2, h = lane >> 4;
                    const uint32_t base = stage + r * 128 + h * 4;
                    __half *to = planes[0] + (rows + jc + h) * p.ldm + i0 + r;
                    const long long step = 2LL * p.ldm, rest = SPLIT ? planes[1] - planes[0] : 0;
                    const bool in = i0 + r < p.m;
                    const int left = p.m - jc - h;
#pragma unroll
                    for (int n = 0; n < 16; n += 4) {
                        float v0[4], v1[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t c = ((n + x) >> 1) ^ (r & 7), low = ((n + x) & 1) * 8;
                            v0[x] = lds_f1(base + c * 16 + low);
                            v1[x] = lds_f1(base + 128 + (c ^ 1) * 16 + low);
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if (in && 2 * (n + x) < left) {
                                const __half2 b = __floats2half2_rn(v0[x], v1[x]);
                                *reinterpret_cast<__half2 *>(to) = b;
                                if (SPLIT) {
                                    const float2 w = __half22float2(b);
                                    *reinterpret_cast<__half2 *>(to + rest) = __floats2half2_rn(v0[x] - w.x, v1[x] - w.y);
                                }
                            }
                            to += step;
                        }
                    }
                } else if (i0 + lane < p.m) {
                    const long long to = mat * p.stride_o + jc * p.ldo + i0 + lane;
#pragma unroll 8
                    for (int c = 0; c < 32; ++c) {
                        if (jc + c >= p.n) break;
                        const float v = lds_f1(at(lane, c >> 2) + (c & 3) * 4);
                        if (p.o_bf16)
                            static_cast<__nv_bfloat16 *>(p.o)[to + c * p.ldo] = __float2bfloat16_rn(v);
                        else
                            static_cast<float *>(p.o)[to + c * p.ldo] = v;
                    }
                }
                __syncwarp();
            };
            if (SPLIT) {
                uint32_t sum[UNITS][16];
                for (int seg0 = 0; seg0 < p.kt; seg0 += SEG) {
                    if (UNITS == 2 && seg0 + SEG >= p.kt) fetch(0);
                    if (!await()) break;
#pragma unroll
                    for (int k = 0; k < UNITS; k += 2) {
                        if (k >= 2 * mine) continue;
                        const int unit = 2 * k + (narrow ? 0 : 2 * half);
                        if (seg0 == 0) {
                            load(unit, sum[k]);
                            load(unit + 1, sum[k + 1]);
                        } else {
                            constexpr int AT_ONCE = UNITS > 4 ? 1 : 2;  // as registers allow
#pragma unroll
                            for (int n = 0; n < 2; n += AT_ONCE) {
                                uint32_t v[AT_ONCE][16];
#pragma unroll
                                for (int i = 0; i < AT_ONCE; ++i) load(unit + n + i, v[i]);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        sum[k + n + i][c] = __float_as_uint(__uint_as_float(sum[k + n + i][c]) +
                                                                            __uint_as_float(v[i][c]));
                            }
                        }
                    }
                    tmem_wait_ld();
                    release();
                }
                if (!ok) break;
                // one body for all chunks: unrolled, it spills
#pragma unroll 1
                for (int k = 0; k < mine; ++k) {
#pragma unroll
                    for (int n = 0; n < UNITS / 2; ++n)
                        if (k == n) turn(sum[2 * n], sum[2 * n + 1]);
                    if (UNITS > 2) fetch(k);
                    finish(k);
                }
            } else {
                fetch(0);
                if (!await()) break;
                uint32_t v[2][16];
#pragma unroll 1
                for (int k = 0; k == 0 || k < mine; ++k) {
                    if (k < mine) {
                        const int unit = narrow ? 0 : 4 * k + 2 * half;
                        load(unit, v[0]);
                        load(unit + 1, v[1]);
                        tmem_wait_ld();
                    }
                    if (k + 1 >= mine) release();
                    if (k < mine) {
                        turn(v[0], v[1]);
                        finish(k);
                        if (k + 1 < mine) fetch(k + 1);
                    }
                }
            }
            __syncwarp();
        }
    }

    tc_fence_before_sync();
    __syncwarp();
    if (CG == 2)
        cluster_sync();  // no CTA leaves while its peer may still target its shared memory
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if (CG == 2)
            tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else
            tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------ norm and start

constexpr int NORM_THREADS = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of a row.
__device__ __forceinline__ void load_vec(const float *src, float (&x)[4])
{
    const float4 v = *reinterpret_cast<const float4 *>(src);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *src, float (&x)[8])
{
    const uint4 v = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ double power_of_two(int k)  // |k| < 1022
{
    return __longlong_as_double(static_cast<long long>(k + 1023) << 52);
}

// From the sum of squares of a matrix: the factor of its first products, the power
// of two that makes Y (two factors, whose product may leave FP32's range), and X's.  FP64 operations
// are slow here (sqrt, division and frexp took 2 us of a call): FP32 results with
// one correction each.
__device__ void write_factors(double sum, double eps, float *f)
{
    // |G| 2^e in [1, 2); 1 / ((|G| + eps) 2^e) = rest 2^-down, rest <= 2, down > 0 only where eps outweighs |G|
    int e = 0, down = 0;
    float rest = 1.0f;
    if (!(sum < INFINITY)) {
        rest = __int_as_float(0x7fffffff);  // NaN
    } else if (sum > 0.0) {
        int two = static_cast<int>(__double_as_longlong(sum) >> 52) - 1023;  // sums of FP32 squares are no FP64 denormals
        two -= two & 1;
        e = -(two / 2);
        const double g = sum * power_of_two(-two);  // in [1, 4)
        const float root = sqrtf(static_cast<float>(g));
        const double r = root, near = r + 0.5f * static_cast<float>(fma(-r, r, g)) / root;
        double h = near + eps * power_of_two(e);
        if (h > 4.0) {
            const int q = static_cast<int>(__double_as_longlong(h) >> 52) - 1023;
            h *= 0.5 * power_of_two(-q);
            down = q + 1;
        }
        rest = 1.0f / static_cast<float>(h);
        rest = fmaf(rest, static_cast<float>(fma(-h, static_cast<double>(rest), 1.0)), rest);
    }
    const int up = e + SCALE_X_LOG, up0 = max(-126, min(126, up));
    f[kFactorRest] = rest;
    f[kFactorUp0] = ldexpf(1.0f, up0);
    f[kFactorUp1] = ldexpf(1.0f, max(-126, min(126, up - up0)));
    f[kFactorLog] = static_cast<float>(SCALE_X_LOG + down);
    f[kFactorMost] = rest * 8192.0f;  // of rest Y
    f[kFactorLog + 1] = f[kFactorMost + 1] = 0.0f;
}

// The sum of squares of rows r0 .. r1 - 1, by a whole CTA.  A thread adds in FP32,
// the threads in FP64.  Where squares would leave FP32 (largest magnitude above
// 2^50 or below 2^-40) the rows are summed again, scaled by a power of two.
template <typename T>
__device__ double squares(const T *base, long long ldg, int r0, int r1, int cols, bool vec)
{
    constexpr int N = 16 / sizeof(T);
    __shared__ double sums[NORM_THREADS / 32];
    __shared__ float tops[NORM_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float scale = 1.0f;
    for (int pass = 0;; ++pass) {
        float top = 0.0f;
        double total = 0.0;
        for (int r = r0 + warp; r < r1; r += NORM_THREADS / 32) {
            const T *row = base + r * ldg;
            for (int c0 = 0; c0 < cols; c0 += 32 * 64) {  // 64 additions in FP32 at a time
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const int c1 = min(cols, c0 + 32 * 64);
                const auto add = [&](float x, int k) {
                    x *= scale;
                    top = fmaxf(top, fabsf(x));
                    s[k & 3] = fmaf(x, x, s[k & 3]);
                };
                int c = c0 + lane * N;
                if (vec) {
#pragma unroll 4
                    for (; c + N <= c1; c += 32 * N) {
                        float x[N];
                        load_vec(row + c, x);
#pragma unroll
                        for (int k = 0; k < N; ++k) add(x[k], k);
                    }
                    for (int k = 0; k < N && c + k < c1; ++k) add(to_f32(row[c + k]), k);
                } else {
#pragma unroll 8
                    for (c = c0 + lane; c < c1; c += 32) add(to_f32(row[c]), 0);
                }
                total += static_cast<double>((s[0] + s[1]) + (s[2] + s[3]));
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, d);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        }
        if (lane == 0) {
            sums[warp] = total;
            tops[warp] = top;
        }
        __syncthreads();
        total = 0.0;
        top = 0.0f;
        for (int w = 0; w < NORM_THREADS / 32; ++w) {
            total += sums[w];
            top = fmaxf(top, tops[w]);
        }
        __syncthreads();
        const bool again = pass == 0 && top > 0.0f && top < INFINITY && (top > 0x1p50f || top < 0x1p-40f);
        if (!again) {
            if (scale == 1.0f) return total;
            const double undo = 1.0 / scale;  // a power of two
            return total * undo * undo;
        }
        int e;
        frexpf(top, &e);
        scale = ldexpf(1.0f, max(-126, min(126, -e)));
    }
}

template <typename T>
__global__ void __launch_bounds__(NORM_THREADS)
    norm_kernel(const T *g, long long ldg, long long stride, int rows, int cols, int num_parts, int all, bool vec,
                double *parts)
{
    griddep_wait();
    griddep_launch_dependents();
    const int per = (rows + num_parts - 1) / num_parts;
    for (int u = blockIdx.x; u < all; u += gridDim.x) {
        const long long b = u / num_parts;
        const int part = static_cast<int>(u - b * num_parts);
        const int r0 = min(rows, part * per), r1 = min(rows, r0 + per);
        const double sum = squares(g + b * stride, ldg, r0, r1, cols, vec);
        if (threadIdx.x == 0) parts[u] = sum;
    }
}

// The sum of a matrix's parts, by a warp.
__device__ double sum_of_parts(const double *parts, int num_parts)
{
    double sum = 0.0;
    for (int k = threadIdx.x & 31; k < num_parts; k += 32) sum += parts[k];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

__global__ void factors_kernel(const double *parts, int num_parts, int batch, float eps, float *factors)
{
    griddep_wait();
    griddep_launch_dependents();
    for (long long b = blockIdx.x; b < batch; b += gridDim.x) {
        const double sum = sum_of_parts(parts + b * num_parts, num_parts);
        if (threadIdx.x == 0) write_factors(sum, eps, factors + b * FACTORS);
    }
}

// X in two FP16 numbers from G, turned where rows > cols.  A CTA takes 64 x 64
// elements at a time.  With num_parts > 0 every CTA also makes the matrix's factors
// from the sums of the norm's parts (one part: of the matrix itself), for a launch
// less.
template <typename T>
__global__ void __launch_bounds__(NORM_THREADS)
    start_kernel(const T *g, long long ldg, long long stride, bool vec, int turned, int m, int n, int ldn, int tiles_j,
                 int tiles, int all, __half *x0, __half *x1, const double *parts, int num_parts, float eps, float *factors)
{
    __shared__ float tile[64][65], f[FACTORS];
    griddep_wait();
    griddep_launch_dependents();
    for (int u = blockIdx.x; u < all; u += gridDim.x) {
        if (u != static_cast<int>(blockIdx.x)) __syncthreads();  // the shared arrays have been read
        const long long b = u / tiles;
        const int t = static_cast<int>(u - b * tiles);
        const int i0 = t / tiles_j * 64, j0 = t % tiles_j * 64;
        constexpr int N = 16 / sizeof(T);
        const T *base = g + b * stride;
        // tile[a][c]: row a of G's part (64 x 64), turned on the way out
        const int ga = turned ? j0 : i0, gc = turned ? i0 : j0, rows = turned ? n : m, cols = turned ? m : n;
        if (vec) {
#pragma unroll
            for (int k = threadIdx.x; k < 64 * 64 / N; k += NORM_THREADS) {
                const int a = k / (64 / N), c = k % (64 / N) * N;
                float x[N];
                if (ga + a < rows && gc + c + N <= cols) {
                    load_vec(base + (ga + a) * ldg + gc + c, x);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        x[i] = ga + a < rows && gc + c + i < cols ? to_f32(base[(ga + a) * ldg + gc + c + i]) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < N; ++i) tile[a][c + i] = x[i];
            }
        } else {
#pragma unroll 4
            for (int k = threadIdx.x; k < 64 * 64; k += NORM_THREADS) {
                const int a = k >> 6, c = k & 63;
                tile[a][c] = ga + a < rows && gc + c < cols ? to_f32(base[(ga + a) * ldg + gc + c]) : 0.0f;
            }
        }
        if (num_parts > 0) {
            double sum = 0.0;
            if (num_parts == 1)
                sum = squares(base, ldg, 0, rows, cols, vec);
            else if (threadIdx.x < 32)
                sum = sum_of_parts(parts + b * num_parts, num_parts);
            if (threadIdx.x == 0) {
                write_factors(sum, eps, f);
                if (t == 0)
                    for (int k = 0; k < FACTORS; ++k) factors[b * FACTORS + k] = f[k];
            }
        } else if (threadIdx.x < FACTORS) {
            f[threadIdx.x] = factors[b * FACTORS + threadIdx.x];
        }
        __syncthreads();
        const float s0 = f[kFactorUp0], s1 = f[kFactorUp1];
#pragma unroll
        for (int k = threadIdx.x; k < 64 * 8; k += NORM_THREADS) {
            const int r = k >> 3, c = (k & 7) * 8;  // 16 bytes of X
            if (i0 + r >= m) continue;
            float v[8], rest[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (turned ? tile[c + i][r] : tile[r][c + i]) * s0 * s1;
            const long long at = (b * m + i0 + r) * ldn + j0 + c;
            *reinterpret_cast<uint4 *>(x0 + at) = round8(v, rest);
            if (x1) *reinterpret_cast<uint4 *>(x1 + at) = round8(rest);
        }
    }
}

template <int CG, bool SPLIT, int STEP, int UNITS>
cudaError_t launch_one(const CUtensorMap (&maps)[4], const Params &p, int grid, cudaStream_t stream)
{
    return launch_pdl(ortho_kernel<CG, SPLIT, STEP, UNITS>, grid, THREADS, SMEM_MAX, stream, CG, maps[0], maps[1], maps[2],
                      maps[3], p);
}

int64_t product_tiles(int step, int ctas, int bn, int64_t m, int64_t n)
{
    const int64_t bm = ctas * BP, ti = (m + bm - 1) / bm;
    if (step == kOrthoX) return ti * ((n + bn - 1) / bn);
    return std::max<int64_t>(1, bm / bn) * (ti * (ti + 1) / 2);
}

}  // namespace

size_t ortho_bytes(int64_t m, int64_t n, bool split)
{
    const int64_t ldm = (m + 63) / 64 * 64, ldn = (n + 63) / 64 * 64;
    const int64_t planes = split ? 2 : 1;
    return static_cast<size_t>(4 * m * ldn * 2 + 2 * planes * m * ldm * 2 + 2 * ldm * 4 + ORTHO_PARTS * 8 + ORTHO_FACTORS * 4);
}

void ortho_layout(OrthoBuffers &o, uint8_t *base, bool split)
{
    const size_t xs = static_cast<size_t>(o.batch) * o.m * o.ldn * 2, as = static_cast<size_t>(o.batch) * o.m * o.ldm * 2;
    const auto take = [&](size_t bytes) {  // whole 256 bytes
        uint8_t *at = base;
        base += (bytes + 255) / 256 * 256;
        return at;
    };
    for (auto &x : o.x)
        for (auto &plane : x) plane = take(xs);
    for (int pl = 0; pl < (split ? 2 : 1); ++pl) {
        o.a[pl] = take(as);
        o.b[pl] = take(as);
    }
    o.da = reinterpret_cast<float *>(take(static_cast<size_t>(o.batch) * o.ldm * 4));
    o.db = reinterpret_cast<float *>(take(static_cast<size_t>(o.batch) * o.ldm * 4));
    o.parts = reinterpret_cast<double *>(take(static_cast<size_t>(o.batch) * ORTHO_PARTS * 8));
    o.factors = reinterpret_cast<float *>(take(static_cast<size_t>(o.batch) * ORTHO_FACTORS * 4));
}

template <int CG, int STEP>
static cudaError_t ready_for()
{
    cudaError_t e = cudaSuccess;
    if constexpr (CG == 1 || STEP != kOrthoX) {
        e = kernel_ready<ortho_kernel<CG, false, STEP, 2>>(SMEM_MAX);
        if (e == cudaSuccess) e = kernel_ready<ortho_kernel<CG, true, STEP, 2>>(SMEM_MAX);
    }
    if (e == cudaSuccess) e = kernel_ready<ortho_kernel<CG, false, STEP, 8>>(SMEM_MAX);
    if (e == cudaSuccess) e = kernel_ready<ortho_kernel<CG, true, STEP, 4>>(SMEM_MAX);
    if constexpr (CG == 2 || STEP == kOrthoX)
        if (e == cudaSuccess) e = kernel_ready<ortho_kernel<CG, true, STEP, 8>>(SMEM_MAX);
    return e;
}

template <int CG, int STEP>
static cudaError_t launch_for(bool split, int bn, const CUtensorMap (&maps)[4], const Params &p, int grid,
                              cudaStream_t stream)
{
    if constexpr (CG == 1 || STEP != kOrthoX)  // pairs take 128 columns of X at least
        if (bn == (STEP == kOrthoX ? 64 : 32))
            return split ? launch_one<CG, true, STEP, 2>(maps, p, grid, stream)
                         : launch_one<CG, false, STEP, 2>(maps, p, grid, stream);
    if constexpr (CG == 2 || STEP == kOrthoX)  // a CTA alone takes 128 columns of A and B at most
        if (split && bn > 128) return launch_one<CG, true, STEP, 8>(maps, p, grid, stream);
    if (split) return launch_one<CG, true, STEP, 4>(maps, p, grid, stream);
    return launch_one<CG, false, STEP, 8>(maps, p, grid, stream);
}

cudaError_t prepare_ortho()
{
    cudaError_t e = kernel_ready<norm_kernel<float>>(0);
    if (e == cudaSuccess) e = kernel_ready<norm_kernel<__nv_bfloat16>>(0);
    if (e == cudaSuccess) e = kernel_ready<factors_kernel>(0);
    if (e == cudaSuccess) e = kernel_ready<start_kernel<float>>(0);
    if (e == cudaSuccess) e = kernel_ready<start_kernel<__nv_bfloat16>>(0);
    if (e == cudaSuccess) e = ready_for<1, kOrthoA>();
    if (e == cudaSuccess) e = ready_for<1, kOrthoB>();
    if (e == cudaSuccess) e = ready_for<1, kOrthoX>();
    if (e == cudaSuccess) e = ready_for<2, kOrthoA>();
    if (e == cudaSuccess) e = ready_for<2, kOrthoB>();
    if (e == cudaSuccess) e = ready_for<2, kOrthoX>();
    return e;
}

cudaError_t launch_ortho_start(const OrthoBuffers &w, const OrthoMatrices &u, bool split, int max_ctas,
                               cudaStream_t stream, int *launches)
{
    // one part below 8192 elements: the start sums it up, a launch less
    const int64_t size = int64_t{u.rows} * u.cols;
    const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ORTHO_PARTS, size / 4096)));
    const int es = u.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(u.g) % 16 == 0 && (u.ldg * es) % 16 == 0 && (u.stride_g * es) % 16 == 0;
    const __nv_bfloat16 *gb = static_cast<const __nv_bfloat16 *>(u.g);
    const float *gf = static_cast<const float *>(u.g);
    cudaError_t e = cudaSuccess;
    if (parts > 1) {
        const int all = parts * w.batch, grid = capped(all, max_ctas);
        e = u.bf16 ? launch_pdl(norm_kernel<__nv_bfloat16>, grid, NORM_THREADS, 0, stream, 1, gb, u.ldg, u.stride_g,
                                u.rows, u.cols, parts, all, vec, w.parts)
                   : launch_pdl(norm_kernel<float>, grid, NORM_THREADS, 0, stream, 1, gf, u.ldg, u.stride_g, u.rows,
                                u.cols, parts, all, vec, w.parts);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    const int tiles_j = (w.n + 63) / 64, tiles = (w.m + 63) / 64 * tiles_j;
    const int all = tiles * w.batch, grid = capped(all, max_ctas), turned = u.rows > u.cols;
    __half *x0 = reinterpret_cast<__half *>(w.x[0][0]), *x1 = split ? reinterpret_cast<__half *>(w.x[0][1]) : nullptr;
    const double *sums = w.parts;
    // Factors made by the start's CTAs save a launch of 2 us, but all of them make
    // them.  One step, us, with a launch of their own / in the start: 1152 CTAs (2 of
    // 1536 x 1536) 67.8 / 69.8, 1872 (13 of 520 x 1020) 97.7 / 97.5, 2048 95.0 / 97.4,
    // 4096 141.6 / 145.7, 8192 235 / 244, 32768 (16 of 2048 x 4096) 794 to 812 / 799 to
    // 802.
    int start_parts = parts;
    if (parts > 1 && all > 1024) {
        e = launch_pdl(factors_kernel, capped(w.batch, max_ctas), 32, 0, stream, 1, sums, parts, w.batch, u.eps,
                       w.factors);
        if (e != cudaSuccess) return e;
        ++*launches;
        start_parts = 0;
    }
    e = u.bf16 ? launch_pdl(start_kernel<__nv_bfloat16>, grid, NORM_THREADS, 0, stream, 1, gb, u.ldg, u.stride_g,
                            vec, turned, w.m, w.n, w.ldn, tiles_j, tiles, all, x0, x1, sums, start_parts, u.eps, w.factors)
               : launch_pdl(start_kernel<float>, grid, NORM_THREADS, 0, stream, 1, gf, u.ldg, u.stride_g, vec, turned, w.m,
                            w.n, w.ldn, tiles_j, tiles, all, x0, x1, sums, start_parts, u.eps, w.factors);
    if (e == cudaSuccess) ++*launches;
    return e;
}

// Estimated cycles of each tile, the least wins: a stage takes its MMA
// instructions (bn / 2 cycles each from 64 columns on) or the arrival of its
// bytes (55 a cycle), a tile its stages or its epilogue, a launch its waves.
OrthoTile ortho_pick_tile(int step, bool split, int64_t batch, int64_t m, int64_t n, int sm_count)
{
    const int64_t kt = ((step == kOrthoA ? n : m) + BK - 1) / BK;
    OrthoTile best;
    double best_t = 0;
    for (int ctas = 1; ctas <= 2; ++ctas)
        for (int bn : {32, 64, 128, 256}) {
            if (step != kOrthoX && ctas * BP % bn) continue;      // columns of tiles within their rows' blocks
            if (step == kOrthoX && bn / ctas < 64) continue;      // whole 128-byte column chunks a CTA
            const double mma = bn == 32 ? 40 : bn == 64 ? 48 : bn / 2;
            const int planes = split ? 2 : 1;
            const double stage = std::max(4 * mma * (split ? 3 : 1), planes * (P_BYTES + bn / ctas * 128) / 55.0);
            const double tile = static_cast<double>(kt) * stage, epi =
                600 + bn * (step == kOrthoA ? 10.0 : 14.0) * (split ? bn > 128 ? 4 : 1.5 : 1);
            const double fill = static_cast<double>(batch * product_tiles(step, ctas, bn, m, n) * ctas) / sm_count;
            const double t = (fill <= 1 ? 1 : fill + 0.3) * std::max(tile, epi) + std::min(tile, epi) + (ctas > 1 ? 1500 : 0);
            if (best_t == 0 || t < best_t) {
                best_t = t;
                best.ctas = ctas;
                best.bn = bn;
            }
        }
    return best;
}

cudaError_t launch_ortho_product(const OrthoBuffers &w, const OrthoMatrices &u, const OrthoProduct &r,
                                 const CUtensorMap (&maps)[4], int sm_count, int max_ctas)
{
    const int planes = r.split ? 2 : 1, cg = r.tile.ctas;
    Params p;
    p.m = w.m;
    p.n = w.n;
    p.ldm = w.ldm;
    p.ldn = w.ldn;
    p.batch = w.batch;
    p.bn = r.tile.bn;
    p.tiles_i = (w.m + cg * BP - 1) / (cg * BP);
    const int64_t tiles = product_tiles(r.step, cg, r.tile.bn, w.m, w.n);
    if (tiles * w.batch > INT_MAX / 2) return cudaErrorInvalidValue;
    p.tiles = static_cast<int>(tiles);
    p.q_bytes = r.tile.bn / cg * 128;
    p.stage_bytes = planes * (P_BYTES + p.q_bytes);
    p.stages = std::min(MAX_STAGES, (SMEM_MAX - 1024 - EPI_BYTES - NUM_BARS * 8 - 16) / p.stage_bytes);
    p.kt = ((r.step == kOrthoA ? w.n : w.m) + BK - 1) / BK;
    p.first = r.first;
    p.last = r.last;
    p.has_rest = r.split || !r.first;  // BF16 input is exact in FP16
    p.from = r.from;
    p.ca = r.ca;
    p.cb = r.cb;
    p.cc = r.cc;
    for (int pl = 0; pl < 2; ++pl) {
        p.x[pl] = reinterpret_cast<const __half *>(w.x[r.from][pl]);
        p.x_out[pl] = reinterpret_cast<__half *>(w.x[r.from ^ 1][pl]);
        p.a[pl] = reinterpret_cast<__half *>(w.a[pl]);
        p.b[pl] = reinterpret_cast<__half *>(w.b[pl]);
    }
    p.da = w.da;
    p.db = w.db;
    p.factors = w.factors;
    p.o = u.o;
    p.ldo = u.ldo;
    p.stride_o = u.stride_o;
    p.turned = u.rows > u.cols;
    p.o_bf16 = u.bf16;
    const int es = u.bf16 ? 2 : 4;
    p.o_vec = reinterpret_cast<uintptr_t>(u.o) % 16 == 0 && (u.ldo * es) % 16 == 0 && (u.stride_o * es) % 16 == 0;
    p.status = r.status;
    p.timeout_ns = r.timeout_ns;
    p.debug_drop = r.debug_drop;
    const int64_t slots = std::max(1, (max_ctas > 0 ? std::min(max_ctas, sm_count) : sm_count) / cg);
    const int grid = static_cast<int>(cg * std::min<int64_t>(tiles * w.batch, slots));
    const auto launch = [&](auto pair) {
        constexpr int CG = decltype(pair)::value;
        return r.step == kOrthoA   ? launch_for<CG, kOrthoA>(r.split, r.tile.bn, maps, p, grid, r.stream)
               : r.step == kOrthoB ? launch_for<CG, kOrthoB>(r.split, r.tile.bn, maps, p, grid, r.stream)
                                   : launch_for<CG, kOrthoX>(r.split, r.tile.bn, maps, p, grid, r.stream);
    };
    return cg == 2 ? launch(std::integral_constant<int, 2>()) : launch(std::integral_constant<int, 1>());
}

}  // namespace dg
