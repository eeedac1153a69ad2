// Grouped tensor-core products for sm_103a (tcgen05.mma): C_g = A_g · B_g over
// ragged row groups, C_g = A_g^T · B_g over ragged contractions, with BF16,
// TF32 or microscaled 4-bit (E2M1 x E8M0) operands and FP32 accumulation.
//
// Orientation.  The MMA's M side (128 tensor-memory lanes per CTA) carries the
// index that runs along a row of C ("P", the columns of C), its N side the
// rows of C ("Q").  N can be any multiple of 16 (32 for a CTA pair), so a
// group's last tile shrinks the instruction to the rows that are left, and few
// rows per expert do not pay for 128-row tiles.  In the epilogue a warp holds
// 32 neighbouring columns of C and walks the rows.  Where C's rows start on 16
// bytes the warp turns 16 x 32 elements in shared memory and writes 16 bytes a
// lane; else every store instruction writes 32 neighbouring elements, at any
// pitch and alignment.  Either way a tile ends at its group's last row, and
// rows of the next group are never touched.
//
// Roles, as in the dense tensor-core kernels: warp 0 TMA producer, warp 1 MMA
// issuer, warps 2-9 epilogue (two accumulators, so the epilogue of a tile
// overlaps the next tile's main loop; two warps a scheduler, because one warp
// issues every fourth cycle at best: 4.6 us for a 128 x 256 tile with four
// warps, which set the pace below K = 4096); for 4-bit operands warps 10-12
// regroup the block scales.
//
// Block scales.  A row's scales are contiguous bytes; the tensor core wants,
// for 128 rows and 128 elements of K, one 4-byte word per row, row i in lane
// i % 32 of column i / 32.  A scale warp per 128 rows loads 64 bytes of every
// row (the scales of SUP = 8 ring stages) into registers, regroups them to
// [stage][word][lane][4] in one of two shared-memory slots, and the MMA issuer
// copies a stage's words to tensor memory (tcgen05.cp) ahead of the stage's
// MMAs, in order with them.  Eight stages at a time because the hand-over (a
// proxy fence, and a release at cluster scope from the odd CTA of a pair) takes
// about 1 us: once a stage it set the pace, 395 us for 8192 x 14336 x 4096
// (157 us now).
//
// Long FP32 sums.  The tensor core's FP32 accumulator drops the bits that do
// not fit at every addition, an error that grows with their number (measured,
// normal values, of the result's norm: 1.0e-6 for 64 additions, 4.4e-6 for 256;
// FP32 multiply-adds 2.5e-7 and 6.1e-7).  For FP32 results of BF16 (TF32)
// operands longer than 12 (8) ring stages, 48 (32) additions, the accumulator
// therefore runs over that many stages at a time, and the epilogue warps add
// the segments in registers, rounding to nearest (5e-7 at any K, for a tenth of
// the rate at K = 4096).  A weight gradient takes this form where all its rows
// together are that long, since one group may hold them all: 16 skewed groups
// of 512 rows on average come to 5.6e-7 instead of 6.4e-7 to 1.2e-6, for 247
// instead of 231 us with the input gradient.  The sums are 128 registers a
// thread beside the segment being added, of the 168 that ten warps leave: 20 to
// 28 bytes are spilled.  BF16 results round by 2^-8 afterwards.  Sums of 4-bit
// products are not cut: an addition covers 64 K elements, and where the block
// scales of a row lie within a factor of 16 the sums need no more than 24 bits
// (measured: exact up to K = 16384).  Scales that spread over 2^16 lose as much
// per addition as above: 1.0e-6 of the result's norm at K = 4096, 4.5e-6 at
// 16384, 1.9e-5 at 65536.
//
// Few tiles.  A launch with fewer tiles than SMs and a long contraction runs
// each tile on a cluster of 2, 4 or 8 CTAs, each with its own range of K.  The
// partial tiles stay in shared memory; every CTA of the cluster adds a share of
// the rows over the cluster, in CTA order, and writes them.
//
// Groups.  The offsets stay on the device.  Every CTA builds the running count
// of its launch's tiles per group in shared memory (one load and a block scan,
// beside the barrier set-up) and finds the group of tile u by bisection.
// Offsets that decrease or leave [0, rows] are reported in the status word and
// the launch computes nothing; reads of the offsets are clamped all the same,
// so no tile reads or writes outside the operands.
//
// Ragged contraction.  The k rows of a group start anywhere and end inside a
// stage.  Both operands are read through a view {column, y < BK, z} whose y
// and z both step one row: the box at (y0 = n - BK, z = r) is zero for y < 0,
// whatever lies there, and holds rows r .. r + n - 1 after that.  The order of
// the k rows within a stage is the same for both operands, so zeros may come
// first.
#include <algorithm>
#include <cuda_bf16.h>

#include <climits>
#include <cstdint>
#include <mutex>

#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr int BP = kRaggedP;
constexpr int P_BYTES = BP * 128;  // 128 rows of P x 128 bytes of K
constexpr int MAX_STAGES = 12;
constexpr int TMEM_COLS = 512;
constexpr int NUM_BARS = 2 * MAX_STAGES + 2 + 2 + 2 + 2 + 1;
// Accumulators at tensor-memory columns 0 and ACC1.  For 4-bit operands the
// scales of two stages live at SF_COL, which leaves two accumulators of 224
// rows: 157 us for 8192 x 14336 x 4096, against 165 us with tiles of 256 rows
// whose accumulators share 48 columns that the epilogue frees first.
constexpr int ACC1 = 256, ACC1_MX = 224;
constexpr int SF_COL = 448, SF_COLS = 24;  // per stage: 2 words x 4 (P) and 2 words x 8 (Q) columns
constexpr int SUP = 8;           // ring stages whose scales are handed over together
constexpr int SF_PART = 1024;    // a stage's words of 128 rows
constexpr int EPI_WARPS = 8;
constexpr int EPI_BYTES = EPI_WARPS * 2048;  // a warp's staging: 16 x 32 FP32, or BF16 in half of it
constexpr int WARPS = 2 + EPI_WARPS, WARPS_MX = WARPS + 3;
constexpr int SMEM_MAX = 227 * 1024;

struct Params {
    const long long *offsets;
    int groups, rows, P, Q, K;
    int bn, tiles_p, tiles_q, group_q, split;
    int stages, stage_bytes, q_bytes, table_bytes, sf_parts;
    void *C;
    long long ldc, stride_c;
    int out_bf16, p_chunks, q_chunks;
    int c_vec;  // 1: C is written in pieces of 16 bytes
    // 4-bit operands: scale bytes of P (groups of P rows) and Q, blocks of K
    const uint8_t *scale_p, *scale_q;
    long long lds_p, lds_q;
    int blocks;
    int *status;
    unsigned long long timeout_ns;
    int debug_drop;
};

__device__ __forceinline__ void group_range(const Params &p, int g, int &lo, int &hi)
{
    if (p.offsets == nullptr) {
        lo = 0;
        hi = p.rows;
        return;
    }
    const long long a = *(p.offsets + g), b = *(p.offsets + g + 1), r = p.rows;
    const long long l = a < 0 ? 0 : a > r ? r : a;
    const long long e = b < l ? l : b > r ? r : b;
    lo = static_cast<int>(l);
    hi = static_cast<int>(e);
}

// Whether the offsets rise within [0, rows], and, for ragged rows, table[g] =
// tiles of the groups before g, table[groups] = all tiles.  All threads call
// it; block 0 reports offsets that do not rise, and every block then runs no
// tile.  Threads take contiguous runs of groups; up to NT groups are read once.
template <int NT, bool TABLE>
__device__ bool read_groups(const Params &p, int *table, int *warp_sum)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.groups + NT - 1) / NT;
    const int g0 = min(p.groups, tid * per), g1 = min(p.groups, g0 + per);
    const auto tiles = [&](int g) {
        int lo, hi;
        group_range(p, g, lo, hi);
        return (hi - lo + p.bn - 1) / p.bn * p.tiles_p;
    };
    int sum = 0, bad = 0, last = 0;
    for (int g = g0; g < g1; ++g) {
        if (p.offsets != nullptr) {
            const long long a = *(p.offsets + g), b = *(p.offsets + g + 1);
            if (a < 0 || b < a || b > p.rows) bad = 1;
        }
        if (TABLE) sum += last = tiles(g);
    }
    int inc = sum;
    if (TABLE) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) warp_sum[warp] = inc;
    }
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && tid == 0) atomicCAS(p.status, 0, kStatusBadOffsets);
    if (TABLE) {
        int before = inc - sum;
        for (int w = 0; w < warp; ++w) before += warp_sum[w];
        for (int g = g0; g < g1; ++g) {
            table[g] = before;
            before += per == 1 ? last : tiles(g);
        }
        if (g0 < p.groups && g1 == p.groups) table[p.groups] = before;
    }
    return bad == 0;
}

struct Tile {
    int g;    // group
    int lo;   // its first row
    int cnt;  // its rows
    int pb;   // tile column index (units of ctas * 128 columns of C)
    int q0;   // first row of the tile within the group's C
    int qn;   // rows of the tile
    int ks;   // first ring stage of this CTA's share of the contraction
    int kt;   // its stages
};

// Tile r of a group's tiles_q x tiles_p: bands of group_q tile rows, column by
// column inside a band, so that CTAs running at the same time share panels.
__device__ __forceinline__ void tile_order(const Params &p, int r, int tiles_q, int &qb, int &pb)
{
    const int per = p.group_q * p.tiles_p;
    const int band = r / per;
    const int first = band * p.group_q;
    const int gq = min(tiles_q - first, p.group_q);
    const int rr = r - band * per;
    qb = first + rr % gq;
    pb = rr / gq;
}

template <int BK, bool RAGGED_K>
__device__ __forceinline__ Tile tile_at(const Params &p, const int *table, int u, int krank)
{
    Tile t;
    int r, tiles_q;
    if (RAGGED_K) {
        const int per = p.tiles_p * p.tiles_q;
        t.g = u / per;
        r = u - t.g * per;
        tiles_q = p.tiles_q;
    } else {
        int a = 0, b = p.groups;  // table[a] <= u < table[b]
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (table[m] <= u)
                a = m;
            else
                b = m;
        }
        t.g = a;
        r = u - table[a];
        tiles_q = 0;
    }
    int hi;
    group_range(p, t.g, t.lo, hi);
    t.cnt = hi - t.lo;
    if (!RAGGED_K) tiles_q = (t.cnt + p.bn - 1) / p.bn;
    int qb;
    tile_order(p, r, tiles_q, qb, t.pb);
    t.q0 = qb * p.bn;
    t.qn = min(p.bn, (RAGGED_K ? p.Q : t.cnt) - t.q0);
    t.ks = 0;
    t.kt = ((RAGGED_K ? t.cnt : p.K) + BK - 1) / BK;
    if (p.split > 1) {
        // even shares: 16 scale bytes of 4-bit operands cover two stages
        const int per = ((t.kt + p.split - 1) / p.split + 1) & ~1;
        t.ks = min(t.kt, krank * per);
        t.kt = min(t.kt - t.ks, per);
    }
    return t;
}

// MMA N of a tile: the rows that are left, in the granularity the instruction
// takes.  The MN-major operand of a ragged contraction keeps whole chunks.
template <int CG, bool RAGGED_K>
__device__ __forceinline__ int mma_n(const Params &p, const Tile &t)
{
    constexpr int G = CG == 2 ? 32 : 16;
    return RAGGED_K ? p.bn : (t.qn + G - 1) / G * G;
}

// Stages of a segment of a long FP32 sum.
__host__ __device__ constexpr int seg_stages(int kind) { return kind == kRaggedTf32 ? 8 : 12; }

// SUM: long FP32 sums (see above).
template <int KIND, int CG, bool P_MN, bool RAGGED_K, bool SUM>
__global__ void __launch_bounds__(32 * (KIND == kRaggedMx4 ? WARPS_MX : WARPS), 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, const Params p)
{
    constexpr bool MX = KIND == kRaggedMx4;
    constexpr int SEG = seg_stages(KIND);
    constexpr int THREADS = 32 * (MX ? WARPS_MX : WARPS);
    constexpr int ES = KIND == kRaggedBf16 ? 2 : 4;                 // bytes an element (not for 4-bit)
    constexpr int BK = MX ? 256 : 128 / ES;                         // K elements of a stage
    constexpr int K_STEPS = 4;                                      // MMA instructions of a stage, 32 bytes of K each
    constexpr int CHUNK = 128 / ES;                                 // MN-major: elements of a 128-byte row
    constexpr int BOX_BYTES = BK * 128;                             // MN-major: one chunk of a stage
    constexpr uint32_t MN_LAYOUT = ES == 2 ? kLayoutSw128 : kLayoutSw128Atom32;
    constexpr uint32_t MN_SBO = ES == 2 ? 1024u : 512u;
    constexpr bool Q_MN = RAGGED_K;
    // Instruction descriptor without N.  BF16 / TF32: FP32 accumulator, operand
    // formats, major-ness; 4-bit: E2M1 formats and E8M0 scales (the scale ids
    // are added per instruction).
    constexpr uint32_t FMT = KIND == kRaggedBf16 ? 1u : 2u;
    constexpr uint32_t IDESC = MX ? (1u << 7) | (1u << 10) | (1u << 23) | (static_cast<uint32_t>((CG * BP) >> 4) << 24)
                                  : (1u << 4) | (FMT << 7) | (FMT << 10) | ((P_MN ? 1u : 0u) << 15) |
                                        ((Q_MN ? 1u : 0u) << 16) | (static_cast<uint32_t>((CG * BP) >> 4) << 24);

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_addr + pad;
    const uint32_t ring = static_cast<uint32_t>(p.stages * p.stage_bytes);
    const uint32_t sf_slot = static_cast<uint32_t>(MX ? SUP * p.sf_parts * SF_PART : 0);  // scales of SUP stages
    const uint32_t sf_base = sbase + ring;                                                 // [2]
    const uint32_t epi_base = sf_base + 2 * sf_slot;
    int *table = reinterpret_cast<int *>(smem + ring + 2 * sf_slot + EPI_BYTES);
    const uint32_t bars = epi_base + EPI_BYTES + p.table_bytes;
    const uint32_t full_bar = bars;                       // [stages], used in the even CTA
    const uint32_t empty_bar = full_bar + 8 * MAX_STAGES;  // [stages]
    const uint32_t tfull_bar = empty_bar + 8 * MAX_STAGES;  // [2]
    const uint32_t tempty_bar = tfull_bar + 16;             // [2], used in the even CTA
    const uint32_t sready_bar = tempty_bar + 16;            // [2], scale slot filled, used in the even CTA
    const uint32_t sfree_bar = sready_bar + 16;             // [2], scale slot read
    const uint32_t drain_bar = sfree_bar + 16;
    uint8_t *tail = smem + ring + 2 * sf_slot + EPI_BYTES + p.table_bytes + NUM_BARS * 8;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
    int *warp_sum = reinterpret_cast<int *>(tail + 16);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    // With a split contraction the cluster's CTAs share a tile (CG = 1 only).
    const int krank = CG == 1 && p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int per_unit = CG == 1 ? p.split : CG;
    const int first_unit = blockIdx.x / per_unit;
    const int unit_step = gridDim.x / per_unit;
    const int acc1 = MX ? ACC1_MX : ACC1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, 1);  // the MMA issuer's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar + 8 * b, 1);
            mbar_init(tempty_bar + 8 * b, EPI_WARPS * CG);
            mbar_init(sready_bar + 8 * b, p.sf_parts + (CG == 2 && leader ? 1 : 0));  // scale warps, the odd CTA
            mbar_init(sfree_bar + 8 * b, 1);                 // the MMA issuer's commit
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
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
    if (threadIdx.x == 0 && (RAGGED_K || p.K > 0)) {
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ);
    }
    // Up to here the kernel may overlap the end of the one before it on the
    // stream.  It does not ask for the next one early: a quantisation that
    // starts beside this kernel finds the SMs unevenly free (8 us lost on
    // 8192 x 14336 x 4096).
    griddep_wait();
    const bool groups_ok = read_groups<THREADS, !RAGGED_K>(p, table, warp_sum);
    tc_fence_before_sync();
    if (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const int num_units = !groups_ok ? 0 : RAGGED_K ? p.groups * p.tiles_p * p.tiles_q : table[p.groups];

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            const int q_cta = p.bn / CG;  // rows of Q this CTA stages
            const uint32_t tx = static_cast<uint32_t>(CG * (P_BYTES + p.q_bytes));
            uint32_t it = 0, s = 0, ph = 0;
            bool ok = true;
            for (int u = first_unit; ok && u < num_units; u += unit_step) {
                const Tile t = tile_at<BK, RAGGED_K>(p, table, u, krank);
                const int p0 = (t.pb * CG + static_cast<int>(rank)) * BP;
                const int n_cta = mma_n<CG, RAGGED_K>(p, t) / CG;
                const int qx = (RAGGED_K ? 0 : t.lo) + t.q0 + static_cast<int>(rank) * n_cta;
                for (int kt = 0; kt < t.kt; ++kt, ++it) {
                    if (!mbar_wait(empty_bar + 8 * s, ph ^ 1u, abort_flag, p.status, kWaitProducerEmpty,
                                   p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = full_bar + 8 * s;
                    const uint32_t fb = CG == 2 ? mapa_shared(fb_local, 0) : fb_local;
                    const uint32_t p_st = sbase + s * p.stage_bytes;
                    const uint32_t q_st = p_st + P_BYTES;
                    if (leader) mbar_arrive_expect_tx(fb_local, tx);
                    if (++s == static_cast<uint32_t>(p.stages)) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (p.debug_drop && blockIdx.x == 0 && it == 0) continue;  // bytes that never come
                    if (RAGGED_K) {
                        // zeros, then rows [z, z + n) of the group
                        const int k = (t.ks + kt) * BK;
                        const int n = min(BK, t.cnt - k);
                        const int y = n - BK, z = t.lo + k;
                        if (p.p_chunks) {
                            if (CG == 2)
                                tma_load_4d_pair(p_st, &tmP, fb, 0, y, z, p0 / CHUNK);
                            else
                                tma_load_4d(p_st, &tmP, fb, 0, y, z, p0 / CHUNK);
                        } else {
                            for (int j = 0; j < BP / CHUNK; ++j) {
                                if (CG == 2)
                                    tma_load_3d_pair(p_st + j * BOX_BYTES, &tmP, fb, p0 + j * CHUNK, y, z);
                                else
                                    tma_load_3d(p_st + j * BOX_BYTES, &tmP, fb, p0 + j * CHUNK, y, z);
                            }
                        }
                        if (p.q_chunks) {
                            if (CG == 2)
                                tma_load_4d_pair(q_st, &tmQ, fb, 0, y, z, qx / CHUNK);
                            else
                                tma_load_4d(q_st, &tmQ, fb, 0, y, z, qx / CHUNK);
                        } else {
                            for (int j = 0; j < q_cta / CHUNK; ++j) {
                                if (CG == 2)
                                    tma_load_3d_pair(q_st + j * BOX_BYTES, &tmQ, fb, qx + j * CHUNK, y, z);
                                else
                                    tma_load_3d(q_st + j * BOX_BYTES, &tmQ, fb, qx + j * CHUNK, y, z);
                            }
                        }
                        continue;
                    }
                    const int kx = (t.ks + kt) * (MX ? 128 : BK);  // 4-bit views count bytes
                    if (P_MN) {
                        if (p.p_chunks) {
                            if (CG == 2)
                                tma_load_4d_pair(p_st, &tmP, fb, 0, kx, p0 / CHUNK, t.g);
                            else
                                tma_load_4d(p_st, &tmP, fb, 0, kx, p0 / CHUNK, t.g);
                        } else {
                            for (int j = 0; j < BP / CHUNK; ++j) {
                                if (CG == 2)
                                    tma_load_3d_pair(p_st + j * BOX_BYTES, &tmP, fb, p0 + j * CHUNK, kx, t.g);
                                else
                                    tma_load_3d(p_st + j * BOX_BYTES, &tmP, fb, p0 + j * CHUNK, kx, t.g);
                            }
                        }
                    } else if (CG == 2) {
                        tma_load_3d_pair(p_st, &tmP, fb, kx, p0, t.g);
                    } else {
                        tma_load_3d(p_st, &tmP, fb, kx, p0, t.g);
                    }
                    if (CG == 2)
                        tma_load_2d_pair(q_st, &tmQ, fb, kx, qx);
                    else
                        tma_load_2d(q_st, &tmQ, fb, kx, qx);
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
                } else {
                    // after an abort: leave no copy in flight (the even CTA's
                    // barriers count both CTAs' operand bytes)
                    if (leader) mbar_wait(full_bar + 8 * ds, dph, &dummy, nullptr, kWaitDrain, p.timeout_ns);
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
            uint32_t it = 0, s = 0, ph = 0, acc_it = 0, sup = 0;
            bool ok = true, issued = false;
            for (int u = first_unit; ok && u < num_units; u += unit_step) {
                const Tile t = tile_at<BK, RAGGED_K>(p, table, u, krank);
                const uint32_t idesc = IDESC | (static_cast<uint32_t>(mma_n<CG, RAGGED_K>(p, t) >> 3) << 17);
                for (int seg0 = 0; seg0 == 0 || seg0 < t.kt; seg0 += SUM ? SEG : t.kt, ++acc_it) {
                    const int seg1 = SUM ? min(t.kt, seg0 + SEG) : t.kt;
                    const uint32_t abuf = acc_it & 1u;
                    if (!mbar_wait_warp(tempty_bar + 8 * abuf, ((acc_it >> 1) & 1u) ^ 1u, abort_flag, p.status,
                                        kWaitMmaTmemEmpty, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + abuf * acc1;
                    for (int kt = seg0; kt < seg1; ++kt, ++it) {
                        if (!mbar_wait_warp(full_bar + 8 * s, ph, abort_flag, p.status, kWaitMmaFull, p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        if (MX && kt % SUP == 0 &&
                            !mbar_wait_warp(sready_bar + 8 * (sup & 1u), (sup >> 1) & 1u, abort_flag, p.status,
                                            kWaitMmaScale, p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t p_st = sbase + s * p.stage_bytes;
                        const uint32_t q_st = p_st + P_BYTES;
                        uint64_t pd[K_STEPS], qd[K_STEPS];
    #pragma unroll
                        for (int kk = 0; kk < K_STEPS; ++kk) {
                            const int kr = kk * (32 / ES) * 128;  // MN-major: K rows of an instruction
                            pd[kk] = P_MN ? smem_desc(p_st + kr, BOX_BYTES, MN_SBO, MN_LAYOUT)
                                          : smem_desc(p_st + kk * 32, 16, 1024, kLayoutSw128);
                            qd[kk] = Q_MN ? smem_desc(q_st + kr, BOX_BYTES, MN_SBO, MN_LAYOUT)
                                          : smem_desc(q_st + kk * 32, 16, 1024, kLayoutSw128);
                        }
                        const uint32_t acc0 = kt > seg0 ? 1u : 0u;
                        const uint32_t sf = tmem_base + SF_COL + (it & 1u) * SF_COLS;
                        const uint64_t sfd = smem_desc(
                            sf_base + (sup & 1u) * sf_slot + static_cast<uint32_t>((kt % SUP) * p.sf_parts * SF_PART), 0,
                            128, kLayoutNone);
                        if (elect_one()) {
                            if (MX) {
                                // 512-byte groups: P's two words, then the two words of each 128 rows of Q
    #pragma unroll
                                for (int i = 0; i < 6; ++i) {
                                    const uint32_t dst = i < 2 ? sf + i * 4 : sf + 8 + (i & 1) * 8 + (i >> 2) * 4;
                                    if (i < 4 || p.bn > 128) {
                                        if (CG == 2)
                                            tmem_copy_32x16b_pair(dst, sfd + i * 32);
                                        else
                                            tmem_copy_32x16b(dst, sfd + i * 32);
                                    }
                                }
                            }
    #pragma unroll
                            for (int kk = 0; kk < K_STEPS; ++kk) {
                                const uint32_t acc = kk > 0 ? 1u : acc0;
                                if (MX) {
                                    const uint32_t id = (kk & 1) ? idesc | (2u << 4) | (2u << 29) : idesc;
                                    const uint32_t sp = sf + (kk >> 1) * 4, sq = sf + 8 + (kk >> 1) * 8;
                                    if (CG == 2)
                                        tc_mma_mx4_pair(d_tmem, pd[kk], qd[kk], id, sp, sq, acc);
                                    else
                                        tc_mma_mx4(d_tmem, pd[kk], qd[kk], id, sp, sq, acc);
                                } else if (KIND == kRaggedBf16) {
                                    if (CG == 2)
                                        tc_mma_f16_pair(d_tmem, pd[kk], qd[kk], idesc, acc);
                                    else
                                        tc_mma_f16(d_tmem, pd[kk], qd[kk], idesc, acc);
                                } else {
                                    if (CG == 2)
                                        tc_mma_tf32_pair(d_tmem, pd[kk], qd[kk], idesc, acc);
                                    else
                                        tc_mma_tf32(d_tmem, pd[kk], qd[kk], idesc, acc);
                                }
                            }
                            if (CG == 2)
                                tc_commit_pair_multicast(empty_bar + 8 * s, 0x3);
                            else
                                tc_commit(empty_bar + 8 * s);
                            if (MX && (kt % SUP == SUP - 1 || kt == t.kt - 1)) {
                                if (CG == 2)
                                    tc_commit_pair_multicast(sfree_bar + 8 * (sup & 1u), 0x3);
                                else
                                    tc_commit(sfree_bar + 8 * (sup & 1u));
                            }
                        }
                        __syncwarp();
                        if (MX && (kt % SUP == SUP - 1 || kt == t.kt - 1)) ++sup;
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
                    if (!SUM) {
                        ++acc_it;
                        break;
                    }
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
        } else if (MX) {
            // The odd CTA's scale slots, announced to the issuer: the release
            // at cluster scope takes about 1 us, which the scale warps are
            // spared.
            uint32_t sup = 0;
            bool ok = true;
            for (int u = first_unit; ok && u < num_units; u += unit_step) {
                const int kts = tile_at<BK, RAGGED_K>(p, table, u, krank).kt;
                for (int k0 = 0; k0 < kts; k0 += SUP, ++sup) {
                    if (!mbar_wait_warp(sready_bar + 8 * (sup & 1u), (sup >> 1) & 1u, abort_flag, p.status,
                                        kWaitMmaScale, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(sready_bar + 8 * (sup & 1u), 0));
                    __syncwarp();
                }
            }
        }
    } else if (warp < 2 + EPI_WARPS) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;            // tensor-memory lane quarter
        const int half = (warp - 2) >> 2;  // 0: even chunks of 32 rows of C, 1: odd ones
        const uint32_t stage = epi_base + static_cast<uint32_t>(warp - 2) * 2048;
        uint32_t acc_it = 0;
        bool ok = true;
        for (int u = first_unit; ok && u < num_units; u += unit_step) {
            const Tile t = tile_at<BK, RAGGED_K>(p, table, u, krank);
            const int col0 = (t.pb * CG + static_cast<int>(rank)) * BP + q * 32;  // the warp's first column
            const long long first_row = RAGGED_K ? t.q0 : static_cast<long long>(t.lo) + t.q0;
            const long long base = (RAGGED_K ? t.g * p.stride_c : 0) + first_row * p.ldc + col0;
            const int chunks = (t.qn + 31) / 32;
            const auto await = [&]() {
                const uint32_t abuf = acc_it & 1u;
                ok = mbar_wait_warp(tfull_bar + 8 * abuf, (acc_it >> 1) & 1u, abort_flag, p.status, kWaitEpiTmemFull,
                                    p.timeout_ns);
                tc_fence_after_sync();
                return ok;
            };
            // The accumulator is in registers: hand it back to the MMA warp.
            // Relaxed, because a release would wait for the stores to C of the
            // columns before (weight gradient of 16 experts of 4096 x 2048:
            // 150 us against 125 to 138, both without segments).
            const auto release = [&]() {
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
                if (t.kt > 0) {
                    tmem_load_16cols(
                        tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc_it & 1u) * acc1 + unit * 16, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0u;  // the empty sum
                }
            };
            // 16 rows of C from unit * 16 on, the warp's 32 columns.
            const auto store = [&](int unit, const uint32_t(&v)[16]) {
                if (CG == 1 && p.split > 1) {
                    // this CTA's part of the sum, [row][128 columns], where the ring was
#pragma unroll
                    for (int j = 0; j < 16; ++j) sts_u32(sbase + (unit * 16 + j) * 512 + (q * 32 + lane) * 4, v[j]);
                    return;
                }
                const int n = t.qn - unit * 16;  // rows left
                if (n <= 0 || col0 >= p.P) return;
                const long long at = base + static_cast<long long>(unit * 16) * p.ldc;
                if (!SUM && p.c_vec && p.out_bf16) {
                    // words of two rows' neighbours, [row pair][column], odd
                    // pairs' 16-byte pieces swapped in twos (bank conflicts)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const __nv_bfloat162 w =
                            __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        sts_u32(stage + j * 128 + ((lane * 4) ^ ((j & 1) * 16)),
                                *reinterpret_cast<const uint32_t *>(&w));
                    }
                    __syncwarp();
                    // a lane: eight columns of two rows
                    const int piece = (lane & 3) * 8, r = (lane >> 2) * 2;
                    const uint32_t src = stage + (lane >> 2) * 128 + piece * 4;
                    const uint32_t swap = ((lane >> 2) & 1) * 16;
                    const uint4 a = lds_u4(src + swap), b = lds_u4(src + (16 - swap));
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.C) + at + r * p.ldc + piece;
                    if (col0 + piece < p.P) {
                        if (r < n)
                            *reinterpret_cast<uint4 *>(out) =
                                make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                           __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
                        if (r + 1 < n)
                            *reinterpret_cast<uint4 *>(out + p.ldc) =
                                make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                           __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
                    }
                    __syncwarp();
                } else if (p.c_vec) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) sts_u32(stage + j * 128 + lane * 4, v[j]);
                    __syncwarp();
                    const int piece = (lane & 7) * 4;
                    float *out = static_cast<float *>(p.C) + at + (lane >> 3) * p.ldc + piece;
#pragma unroll
                    for (int i = 0; i < 4; ++i, out += 4 * p.ldc) {
                        const int r = i * 4 + (lane >> 3);
                        const uint4 x = lds_u4(stage + r * 128 + piece * 4);
                        if (r < n && col0 + piece < p.P) *reinterpret_cast<uint4 *>(out) = x;
                    }
                    __syncwarp();
                } else if (col0 + lane < p.P) {
                    if (!SUM && p.out_bf16) {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.C) + at + lane;
#pragma unroll
                        for (int j = 0; j < 16; ++j, out += p.ldc)
                            if (j < n) *out = __float2bfloat16_rn(__uint_as_float(v[j]));
                    } else {
                        float *out = static_cast<float *>(p.C) + at + lane;
#pragma unroll
                        for (int j = 0; j < 16; ++j, out += p.ldc)
                            if (j < n) *out = __uint_as_float(v[j]);
                    }
                }
            };
            // This warp's chunks of 32 rows: half, half + 2, ...; unit k of them
            // is 16 rows.
            const int mine = (chunks + 1 - half) / 2;
            const auto unit_of = [&](int k) { return 4 * (k >> 1) + 2 * half + (k & 1); };
            if (SUM) {
                uint32_t sum[8][16];
                for (int seg0 = 0; seg0 == 0 || seg0 < t.kt; seg0 += SEG) {
                    if (!await()) break;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k >= 2 * mine) break;
                        if (seg0 == 0) {
                            load(unit_of(k), sum[k]);
                        } else {
                            uint32_t v[16];
                            load(unit_of(k), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                sum[k][j] = __float_as_uint(__uint_as_float(sum[k][j]) + __uint_as_float(v[j]));
                        }
                    }
                    tmem_wait_ld();
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < 2 * mine) store(unit_of(k), sum[k]);
            } else {
                if (!await()) break;
                uint32_t v[2][16];
#pragma unroll 1
                for (int k = 0; k == 0 || k < 2 * mine; k += 2) {
                    if (k < 2 * mine) {
                        load(unit_of(k), v[0]);
                        load(unit_of(k + 1), v[1]);
                        tmem_wait_ld();
                    }
                    if (k + 2 >= 2 * mine) release();
                    if (k < 2 * mine) {
                        store(unit_of(k), v[0]);
                        store(unit_of(k + 1), v[1]);
                    }
                }
            }
            __syncwarp();
        }
    } else if (MX && p.K > 0 && (warp - 2 - EPI_WARPS - 1) * 128 < p.bn) {
        // ------------------------------------------------------ block scales
        // The first: P's rows; the others: 128 rows of Q each.  Out-of-range
        // rows and blocks get scale byte 0 (their codes are zero).
        // The loads of the next hand-over are issued once the present one is
        // announced (in front of its fence, which waits for them, they cost
        // 166 instead of 157 us on 8192 x 14336 x 4096) and land while the
        // warp waits for a free slot.
        const int part = warp - 2 - EPI_WARPS;
        const long long ld = part == 0 ? p.lds_p : p.lds_q;
        int u = first_unit, k0 = 0, kts = 0, first = 0, limit = 0, blocks = 0;
        const uint8_t *base = nullptr;
        // Lane l loads 16-byte piece l / 8 of rows l % 8, l % 8 + 8, ...: eight
        // rows' 64 bytes an instruction, whole sectors; eight lanes then store
        // 128 contiguous bytes.
        const int piece = lane >> 3, row8 = lane & 7;
        uint4 r[16];
        const auto tile = [&]() {
            if (u >= num_units) return;
            const Tile t = tile_at<BK, RAGGED_K>(p, table, u, krank);
            kts = t.kt;
            first = (part == 0 ? (t.pb * CG + static_cast<int>(rank)) * BP : t.q0 + (part - 1) * 128) + row8;
            limit = part == 0 ? p.P : t.cnt;
            base = (part == 0 ? p.scale_p + static_cast<long long>(t.g) * p.P * ld
                              : p.scale_q + static_cast<long long>(t.lo) * ld) +
                   first * ld + t.ks * 8 + piece * 16;
            blocks = p.blocks - t.ks * 8;
        };
        const auto fetch = [&]() {
            const bool in_k = u < num_units && k0 * 8 + piece * 16 < blocks;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                r[i] = make_uint4(0u, 0u, 0u, 0u);
                if (in_k && first + 8 * i < limit)
                    r[i] = *reinterpret_cast<const uint4 *>(base + 8 * i * ld + k0 * 8);
            }
        };
        tile();
        fetch();
        for (uint32_t sup = 0; u < num_units; ++sup) {
            const uint32_t slot = sup & 1u;
            if (!mbar_wait_warp(sfree_bar + 8 * slot, ((sup >> 1) & 1u) ^ 1u, abort_flag, p.status, kWaitScaleEmpty,
                                p.timeout_ns))
                break;
            // word w of the piece: stage 2 * piece + w / 2, word w % 2
            const uint32_t stage_step = static_cast<uint32_t>(p.sf_parts * SF_PART);
            const uint32_t dst = sf_base + slot * sf_slot + part * SF_PART + 2 * piece * stage_step + row8 * 16;
            const int left = blocks - k0 * 8 - piece * 16;  // blocks of K from the piece on
            const auto keep = [&](uint32_t w, int n) {        // the first n bytes of a word
                return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
            };
            if (left < 16)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    r[i] = make_uint4(keep(r[i].x, left), keep(r[i].y, left - 4), keep(r[i].z, left - 8),
                                      keep(r[i].w, left - 12));
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // rows 8 i + row8 + (0, 32, 64, 96)
                const uint32_t at = dst + i * 128;
                sts_u4(at, make_uint4(r[i].x, r[i + 4].x, r[i + 8].x, r[i + 12].x));
                sts_u4(at + 512, make_uint4(r[i].y, r[i + 4].y, r[i + 8].y, r[i + 12].y));
                sts_u4(at + stage_step, make_uint4(r[i].z, r[i + 4].z, r[i + 8].z, r[i + 12].z));
                sts_u4(at + stage_step + 512, make_uint4(r[i].w, r[i + 4].w, r[i + 8].w, r[i + 12].w));
            }
            k0 += SUP;
            if (k0 >= kts) {
                k0 = 0;
                u += unit_step;
                tile();
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(sready_bar + 8 * slot);
            fetch();
        }
    }

    if (CG == 1 && p.split > 1) {
        // Add the cluster's partial tiles, rows krank, krank + split, ... here,
        // four columns a thread.
        __syncwarp();
        cluster_sync();
        if (first_unit < num_units) {
            const Tile t = tile_at<BK, RAGGED_K>(p, table, first_unit, krank);
            const long long first_row = RAGGED_K ? t.q0 : static_cast<long long>(t.lo) + t.q0;
            const int piece = (threadIdx.x & 31) * 4;
            const int col = t.pb * BP + piece;
            for (int j = krank + p.split * warp; j < t.qn && col < p.P; j += p.split * (THREADS / 32)) {
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int r = 0; r < p.split; ++r) {
                    const float4 y = lds_cluster_f4(mapa_shared(sbase + j * 512 + piece * 4, r));
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                const long long at = (RAGGED_K ? t.g * p.stride_c : 0) + (first_row + j) * p.ldc + col;
                const float v[4] = {x.x, x.y, x.z, x.w};
                if (p.out_bf16) {
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.C) + at;
                    if (p.c_vec) {
                        const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
                        *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(w);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + i < p.P) out[i] = __float2bfloat16_rn(v[i]);
                    }
                } else {
                    float *out = static_cast<float *>(p.C) + at;
                    if (p.c_vec) {
                        *reinterpret_cast<float4 *>(out) = x;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + i < p.P) out[i] = v[i];
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its part
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

// A launch of its own, about 3 us where nothing is wrong: in the weight
// gradient's epilogue, as a loop over the tiles left unwritten, it cost every
// such call 2 to 3 % (16 experts of 4096 x 2048: 147.1 -> 149.8 to 153.3 us in
// five forms, by the compiler's choice of spills alone), and a fill in front of
// the call 65 us.
__global__ void __launch_bounds__(256)
    nan_on_error_kernel(const long long *offsets, int groups, long long rows, int M, int N, void *C, long long ldc,
                        long long stride_c, int out_bf16, const int *status)
{
    griddep_wait();
    int bad = (*status & kStatusTimeout) != 0 ? 1 : 0;
    for (int g = threadIdx.x; g < groups; g += blockDim.x)
        if (offsets[g] < 0 || offsets[g + 1] < offsets[g] || offsets[g + 1] > rows) bad = 1;
    if (!__syncthreads_or(bad)) return;
    const float nan = __int_as_float(0x7fffffff);
    const int lane = threadIdx.x & 31;
    const long long all = static_cast<long long>(groups) * M;
    for (long long r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < all; r += gridDim.x * 8LL) {
        const long long g = r / M, at = g * stride_c + (r - g * M) * ldc;
        for (int c = lane; c < N; c += 32) {
            if (out_bf16)
                static_cast<__nv_bfloat16 *>(C)[at + c] = __float2bfloat16_rn(nan);
            else
                static_cast<float *>(C)[at + c] = nan;
        }
    }
}

template <int KIND, int CG, bool P_MN, bool RK, bool SUM>
cudaError_t set_attrs()
{
    return cudaFuncSetAttribute(ragged_kernel<KIND, CG, P_MN, RK, SUM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM_MAX);
}

template <int KIND, int CG, bool P_MN, bool RK, bool SUM>
cudaError_t launch_one(const CUtensorMap &tmP, const CUtensorMap &tmQ, const Params &p, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * (KIND == kRaggedMx4 ? WARPS_MX : WARPS));
    cfg.dynamicSmemBytes = SMEM_MAX;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG == 1 ? p.split : CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = attr[1].val.clusterDim.x > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ragged_kernel<KIND, CG, P_MN, RK, SUM>, tmP, tmQ, p);
}

// The instantiation for a launch (op: apply<kind, ctas, P MN-major, ragged K, long FP32 sums>).
template <int KIND, int CG, typename Op>
cudaError_t dispatch_form(bool p_mn, bool ragged_k, bool sum, const Op &op)
{
    if (ragged_k) return sum ? op.template apply<KIND, CG, true, true, true>() : op.template apply<KIND, CG, true, true, false>();
    if (p_mn) return sum ? op.template apply<KIND, CG, true, false, true>() : op.template apply<KIND, CG, true, false, false>();
    return sum ? op.template apply<KIND, CG, false, false, true>() : op.template apply<KIND, CG, false, false, false>();
}

template <typename Op>
cudaError_t dispatch(int kind, int ctas, bool p_mn, bool ragged_k, bool sum, const Op &op)
{
    if (kind == kRaggedMx4)
        return ctas == 2 ? op.template apply<kRaggedMx4, 2, false, false, false>()
                         : op.template apply<kRaggedMx4, 1, false, false, false>();
    if (kind == kRaggedTf32)
        return ctas == 2 ? dispatch_form<kRaggedTf32, 2>(p_mn, ragged_k, sum, op)
                         : dispatch_form<kRaggedTf32, 1>(p_mn, ragged_k, sum, op);
    return ctas == 2 ? dispatch_form<kRaggedBf16, 2>(p_mn, ragged_k, sum, op)
                     : dispatch_form<kRaggedBf16, 1>(p_mn, ragged_k, sum, op);
}

struct SetAttrs {
    template <int K, int CG, bool P, bool R, bool S>
    cudaError_t apply() const
    {
        return set_attrs<K, CG, P, R, S>();
    }
};

struct Launch {
    const CUtensorMap &tmP, &tmQ;
    const Params &p;
    int grid;
    cudaStream_t stream;
    template <int K, int CG, bool P, bool R, bool S>
    cudaError_t apply() const
    {
        return launch_one<K, CG, P, R, S>(tmP, tmQ, p, grid, stream);
    }
};

// Tiles of a launch at most (row offsets are on the device): every busy group
// adds at most one partial tile.
int64_t max_units(bool ragged_k, int64_t rows, int64_t groups, int64_t P, int64_t Q, int ctas, int bn)
{
    const int64_t tiles_q =
        ragged_k ? (Q + bn - 1) / bn * groups : (rows + bn - 1) / bn + std::max<int64_t>(0, std::min(groups, rows) - 1);
    return std::max<int64_t>(1, tiles_q * ((P + ctas * BP - 1) / (ctas * BP)));
}

// Clusters of 2, 4 and 8 CTAs that run at the same time (the SMs of a cluster
// share a GPC, so fewer than SMs / size); filled in by the first prepare_ragged
// and not changed after that.
int g_clusters[3] = {};
std::mutex g_prepare;

int max_clusters(int split) { return g_clusters[split == 2 ? 0 : split == 4 ? 1 : 2]; }

cudaError_t query_clusters(int split, int *out)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(32 * WARPS_MX);
    cfg.dynamicSmemBytes = SMEM_MAX;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(out, ragged_kernel<kRaggedMx4, 1, false, false, false>, &cfg);
}

}  // namespace

cudaError_t prepare_ragged()
{
    const std::lock_guard<std::mutex> lock(g_prepare);
    cudaError_t e = cudaSuccess;
    for (int kind : {kRaggedBf16, kRaggedTf32, kRaggedMx4})
        for (int ctas = 1; ctas <= 2; ++ctas)
            for (int form = 0; form < 3; ++form)
                for (bool sum : {false, true})
                    if (e == cudaSuccess) e = dispatch(kind, ctas, form > 0, form == 2, sum, SetAttrs());
    for (int i = 0; i < 3; ++i)
        if (e == cudaSuccess && g_clusters[i] == 0) e = query_clusters(2 << i, &g_clusters[i]);
    return e;
}

bool ragged_tile_ok(int split, int ctas, int bn)
{
    if (!(bn == 32 || bn == 64 || bn == 128 || bn == 224 || bn == 256)) return false;
    if (split <= 1) return split == 0 && (ctas == 1 || ctas == 2);
    return (split == 2 || split == 4 || split == 8) && ctas == 1 && bn <= 128;
}

// Estimated time of each tile in cycles; the least wins.  A ring stage takes
// its four MMA instructions (measured: 128 cycles at N = 256, 64 at 128, 48 at
// 64, 40 at 32) or the arrival of its bytes (55 a cycle and SM measured),
// whichever is longer; a tile its stages (and for 4-bit pairs 3000 cycles: the
// scales' hand-over between the CTAs) or its epilogue (12 cycles a row); a
// launch the waves of tiles, one epilogue and 3 us, and at least its traffic at
// 6.4 TB/s.  The type of C does not enter, so that a BF16 result is the FP32
// result rounded where that is not summed in segments.  The number of TMA boxes
// of a stage does not enter either (one, or one per 128-byte chunk where a width
// is no multiple of the chunk): 13 + 10 us for the TF32 gradients of 2011 rows and
// 13 experts of 1020 x 520, which take 24 + 27.
RaggedTile ragged_pick_tile(int kind, bool ragged_k, int64_t rows, int groups, int64_t P, int64_t Q, int64_t K,
                            int sm_count, bool may_split)
{
    const double es = kind == kRaggedMx4 ? 17.0 / 32 : kind == kRaggedTf32 ? 4 : 2, eo = ragged_k ? 4 : 2;
    const double busy = static_cast<double>(std::max<int64_t>(1, std::min<int64_t>(groups, rows)));
    const double per_group = static_cast<double>(rows) / busy;
    const int bk = ragged_bk(kind);
    const int64_t k_len = ragged_k ? (rows + groups - 1) / groups : K;
    const int64_t kt = std::max<int64_t>(1, (k_len + bk - 1) / bk);
    const double bytes = ragged_k ? double(rows) * (P + Q) * es + double(groups) * P * Q * eo
                                  : double(rows) * K * es + busy * P * K * es + double(rows) * P * eo;
    RaggedTile best;
    double best_t = 0;
    for (int ctas = 1; ctas <= 2; ++ctas)
        for (int bn : {32, 64, 128, kind == kRaggedMx4 ? ACC1_MX : 256})
            for (int split = 1; split <= 8; split *= 2) {
                if (ragged_k && bn < 128) continue;  // whole 128-byte column chunks per CTA
                const int64_t units = max_units(ragged_k, rows, groups, P, Q, ctas, bn);
                if (split > 1 && (!may_split || ctas > 1 || bn > 128 || units > max_clusters(split) || units * split > sm_count ||
                                  kt < 4 * split))
                    continue;
                const double mma = bn == 32 ? 40 : bn == 64 ? 48 : bn / 2;
                const double stage = std::max(4 * mma, (P_BYTES + bn / ctas * 128) / 55.0) * (kind == kRaggedMx4 ? 1.1 : 1);
                const double tiles_p = static_cast<double>((P + ctas * BP - 1) / (ctas * BP));
                const double tiles_q = ragged_k     ? double(groups) * ((Q + bn - 1) / bn)
                                       : busy > 1.5 ? busy * std::max(1.0, per_group / bn + 0.5)
                                                    : double((rows + bn - 1) / bn);
                const double tile = static_cast<double>((kt + split - 1) / split) * stage +
                                    (kind == kRaggedMx4 && ctas > 1 ? 3000 : 0);
                const double epi = 600 + bn * 12.0;
                const double fill = tiles_q * tiles_p * ctas * split / sm_count;
                const double run = (fill <= 1 ? 1 : fill + 0.3) * std::max(tile, epi) + std::min(tile, epi) +
                                   (split > 1 || ctas > 1 ? 1500 : 0);
                const double mem = bytes / 3370;
                const double t = std::max(run, mem) + 0.1 * std::min(run, mem) + 6000;
                if (best.bn == 0 || t < best_t) {
                    best_t = t;
                    best.ctas = ctas;
                    best.bn = bn;
                    best.split = split;
                }
            }
    return best;
}

cudaError_t launch_ragged(int kind, bool ragged_k, bool p_mn, const RaggedTile &t, const CUtensorMap &tmP,
                          const CUtensorMap &tmQ, const RaggedArgs &a, int sm_count, int max_ctas)
{
    Params p;
    p.offsets = reinterpret_cast<const long long *>(a.offsets);
    p.groups = a.groups;
    p.rows = a.rows;
    p.P = a.P;
    p.Q = a.Q;
    p.K = a.K;
    p.bn = t.bn;
    p.tiles_p = (a.P + t.ctas * BP - 1) / (t.ctas * BP);
    p.tiles_q = ragged_k ? (a.Q + t.bn - 1) / t.bn : 0;
    p.split = t.split;
    p.q_bytes = t.bn / t.ctas * 128;
    p.stage_bytes = P_BYTES + p.q_bytes;
    p.sf_parts = 1 + (t.bn + 127) / 128;
    p.table_bytes = ragged_k ? 0 : (4 * (a.groups + 1) + 15) / 16 * 16;
    const int sf_bytes = kind == kRaggedMx4 ? 2 * SUP * p.sf_parts * SF_PART : 0;
    const int fixed = 1024 + sf_bytes + EPI_BYTES + p.table_bytes + NUM_BARS * 8 + 16 + 64;
    p.stages = std::min(MAX_STAGES, (SMEM_MAX - fixed) / p.stage_bytes);
    p.C = a.C;
    p.ldc = a.ldc;
    p.stride_c = a.stride_c;
    p.out_bf16 = a.out_bf16;
    // 16-byte pieces of C: aligned rows that hold whole pieces
    const int eo = a.out_bf16 ? 2 : 4;
    p.c_vec = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && (a.ldc * eo) % 16 == 0 && (a.stride_c * eo) % 16 == 0 &&
              (int64_t{a.P} * eo) % 16 == 0;
    p.p_chunks = a.p_chunks;
    p.q_chunks = a.q_chunks;
    p.scale_p = a.scale_p;
    p.scale_q = a.scale_q;
    p.lds_p = a.lds_p;
    p.lds_q = a.lds_q;
    p.blocks = (a.K + kRaggedBlock - 1) / kRaggedBlock;
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    p.debug_drop = a.debug_drop;
    p.group_q = 16;
    // A persistent grid; one cluster a tile where the contraction is split.
    const int64_t units = max_units(ragged_k, a.rows, a.groups, a.P, a.Q, t.ctas, t.bn);
    const int64_t slots = std::max(1, (max_ctas > 0 ? std::min(max_ctas, sm_count) : sm_count) / t.ctas);
    const int64_t grid = t.split > 1 ? units * t.split : t.ctas * std::min(units, slots);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    // Stages a CTA adds up: of the longest group there can be, for a ragged
    // contraction, whose offsets only the device knows.
    const int bk = ragged_bk(kind);
    const int64_t k_len = ragged_k ? a.rows : a.K;
    const int64_t seg = int64_t{seg_stages(kind)} * t.split;
    const bool sum = a.out_bf16 == 0 && (k_len + bk - 1) / bk > seg;
    return dispatch(kind, t.ctas, p_mn, ragged_k, sum, Launch{tmP, tmQ, p, static_cast<int>(grid), a.stream});
}

cudaError_t launch_nan_on_error(const RaggedArgs &a, int sm_count)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count);
    cfg.blockDim = dim3(256);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, nan_on_error_kernel, reinterpret_cast<const long long *>(a.offsets), a.groups,
                              static_cast<long long>(a.rows), a.Q, a.P, a.C, static_cast<long long>(a.ldc),
                              static_cast<long long>(a.stride_c), a.out_bf16, static_cast<const int *>(a.status));
}

}  // namespace dg
