// The C ABI of include/gemm_grouped.h and include/gemm_mx4.h: argument checks,
// re-packing of operands TMA cannot address, tensor-map encoding and dispatch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/gemm.h"
#include "../../include/gemm_grouped.h"
#include "../../include/gemm_mx4.h"
#include "gemm_internal.h"
#include "handle.h"
#include "ragged.h"

using dg::cuda_fail;
using dg::fail;
using dg::kMaxDim;
using dg::kMaxLd;
using dg::round_up;

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 37;  // elements from one group's matrix to the next (TMA: below 2^40 bytes)
static_assert(GEMM_GROUPED_MAX_GROUPS == dg::kRaggedMaxGroups, "the header states the kernel's limit");
static_assert(GEMM_MX4_BLOCK == dg::kRaggedBlock, "the header states the format's block");

struct Checker {
    std::string *why;
    int operator()(int code, const char *msg) const
    {
        if (why) *why = msg;
        return code;
    }
};

// Whether rows at this pitch span more elements (or bytes) than any memory
// holds; below that no product of the checks and of the set-up overflows.
bool beyond_memory(int64_t rows, int64_t ld) { return rows > 0 && ld > (int64_t{1} << 44) / rows; }

constexpr const char *kBeyondMemory = "rows times pitch must stay within 2^44";

int check_c(const Checker &bad, const void *C, int64_t ldc, int64_t rows, int64_t N, int c_dtype)
{
    if (!C) return bad(GEMM_ERR_INVALID, "C is NULL");
    if (ldc < N || ldc > kMaxLd) return bad(GEMM_ERR_INVALID, "ldc must satisfy N <= ldc <= 2^36");
    if (beyond_memory(rows, ldc)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    if (reinterpret_cast<uintptr_t>(C) % (c_dtype == GEMM_BF16 ? 2 : 4))
        return bad(GEMM_ERR_ALIGNMENT, "C is not aligned to its element size");
    return GEMM_OK;
}

int check_groups(const Checker &bad, int64_t groups, int64_t rows, const int64_t *offsets)
{
    if (groups < 1 || groups > GEMM_GROUPED_MAX_GROUPS)
        return bad(GEMM_ERR_INVALID, "groups must be in 1..GEMM_GROUPED_MAX_GROUPS");
    if (rows < 0 || rows > kMaxDim) return bad(GEMM_ERR_INVALID, "rows must be in 0..2^31 - 1025");
    if (!offsets) return bad(GEMM_ERR_INVALID, "offsets is NULL");
    if (reinterpret_cast<uintptr_t>(offsets) % 8) return bad(GEMM_ERR_ALIGNMENT, "offsets is not 8-byte aligned");
    return GEMM_OK;
}

int check_types(const Checker &bad, int dtype, int c_dtype)
{
    if (dtype != GEMM_BF16 && dtype != GEMM_TF32)
        return bad(GEMM_ERR_INVALID, "grouped products take dtype GEMM_BF16 or GEMM_TF32");
    if (c_dtype != GEMM_F32 && c_dtype != GEMM_BF16)
        return bad(GEMM_ERR_INVALID, "c_dtype must be GEMM_F32 or GEMM_BF16");
    if (dtype == GEMM_TF32 && c_dtype != GEMM_F32) return bad(GEMM_ERR_INVALID, "GEMM_TF32 writes C as GEMM_F32");
    return GEMM_OK;
}

// Takes GEMM_GROUPED_NAN_ON_ERROR off a c_dtype argument.
bool take_nan_flag(int &c_dtype)
{
    const bool nan = (c_dtype & GEMM_GROUPED_NAN_ON_ERROR) != 0;
    c_dtype &= ~GEMM_GROUPED_NAN_ON_ERROR;
    return nan;
}

// Tiles are counted in 32 bits on the device; `rows_of_c` rows cut into tiles
// of at least 32, plus one per group.
bool too_many_tiles(int64_t rows_of_c, int64_t groups, int64_t cols)
{
    return (rows_of_c / 32 + groups + 1) * ((cols + 127) / 128) >= (int64_t{1} << 31);
}

int check_grouped(int layout_b, int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                  const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b, const void *C,
                  int64_t ldc, int dtype, int c_dtype, std::string *why)
{
    const Checker bad{why};
    if (layout_b != GEMM_B_ROW_MAJOR && layout_b != GEMM_B_COL_MAJOR)
        return bad(GEMM_ERR_INVALID, "layout_b must be GEMM_B_ROW_MAJOR or GEMM_B_COL_MAJOR");
    int rc = check_types(bad, dtype, c_dtype);
    if (rc) return rc;
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxDim) return bad(GEMM_ERR_INVALID, "N and K must be in 0..2^31 - 1025");
    if ((rc = check_groups(bad, groups, rows, offsets))) return rc;
    if (rows == 0 || N == 0) return GEMM_OK;
    if (too_many_tiles(rows, groups, N)) return bad(GEMM_ERR_INVALID, "the product has 2^31 tiles or more");
    if ((rc = check_c(bad, C, ldc, rows, N, c_dtype))) return rc;
    if (K == 0) return GEMM_OK;
    if (!A || !B) return bad(GEMM_ERR_INVALID, "A or B is NULL");
    if (lda < K || lda > kMaxLd) return bad(GEMM_ERR_INVALID, "lda must satisfy K <= lda <= 2^36");
    const int64_t rows_b = layout_b == GEMM_B_ROW_MAJOR ? K : N, cols_b = layout_b == GEMM_B_ROW_MAJOR ? N : K;
    if (ldb < cols_b || ldb > kMaxLd)
        return bad(GEMM_ERR_INVALID, "ldb must be at least a row of B's storage and at most 2^36");
    if (beyond_memory(rows, lda) || beyond_memory(rows_b, ldb)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    if (groups > 1 && (stride_b < (rows_b - 1) * ldb + cols_b || stride_b > kMaxStride))
        return bad(GEMM_ERR_INVALID, "stride_b must reach past a group's matrix and stay within 2^37");
    const uintptr_t es = dtype == GEMM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(A) % es || reinterpret_cast<uintptr_t>(B) % es)
        return bad(GEMM_ERR_ALIGNMENT, "A or B is not aligned to its element size");
    return GEMM_OK;
}

int check_wgrad(int64_t groups, int64_t rows, int64_t M, int64_t N, const int64_t *offsets, const void *A,
                int64_t lda, const void *B, int64_t ldb, const void *C, int64_t ldc, int64_t stride_c, int dtype,
                int c_dtype, std::string *why)
{
    const Checker bad{why};
    int rc = check_types(bad, dtype, c_dtype);
    if (rc) return rc;
    if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return bad(GEMM_ERR_INVALID, "M and N must be in 0..2^31 - 1025");
    if ((rc = check_groups(bad, groups, rows, offsets))) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    if (too_many_tiles(M * groups, groups, N)) return bad(GEMM_ERR_INVALID, "the product has 2^31 tiles or more");
    if ((rc = check_c(bad, C, ldc, M, N, c_dtype))) return rc;
    if (groups > 1 && (stride_c < (M - 1) * ldc + N || stride_c > kMaxStride))
        return bad(GEMM_ERR_INVALID, "stride_c must reach past a group's matrix and stay within 2^37");
    if (rows == 0) return GEMM_OK;
    if (!A || !B) return bad(GEMM_ERR_INVALID, "A or B is NULL");
    if (lda < M || lda > kMaxLd) return bad(GEMM_ERR_INVALID, "lda must satisfy M <= lda <= 2^36");
    if (ldb < N || ldb > kMaxLd) return bad(GEMM_ERR_INVALID, "ldb must satisfy N <= ldb <= 2^36");
    if (beyond_memory(rows, lda) || beyond_memory(rows, ldb)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    const uintptr_t es = dtype == GEMM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(A) % es || reinterpret_cast<uintptr_t>(B) % es)
        return bad(GEMM_ERR_ALIGNMENT, "A or B is not aligned to its element size");
    return GEMM_OK;
}

int check_mx4_operand(const Checker &bad, int64_t rows, int64_t K, const void *codes, int64_t ldq, const void *scales,
                      int64_t lds)
{
    if (!codes || !scales) return bad(GEMM_ERR_INVALID, "codes or scales is NULL");
    const int64_t Kp = round_up(K, GEMM_MX4_BLOCK);
    if (ldq < Kp / 2 || ldq > kMaxLd) return bad(GEMM_ERR_INVALID, "the code pitch must hold a row of codes");
    if (lds < Kp / 32 || lds > kMaxLd) return bad(GEMM_ERR_INVALID, "the scale pitch must hold a row of scales");
    if (reinterpret_cast<uintptr_t>(codes) % 16 || reinterpret_cast<uintptr_t>(scales) % 16 || ldq % 16 || lds % 16)
        return bad(GEMM_ERR_ALIGNMENT, "codes, scales and their pitches must be multiples of 16 bytes");
    if (beyond_memory(rows, ldq) || beyond_memory(rows, lds)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    return GEMM_OK;
}

int check_mx4(int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets, const void *ac,
              int64_t aq, const void *as, int64_t al, const void *bc, int64_t bq, const void *bs, int64_t bl,
              const void *C, int64_t ldc, int c_dtype, bool grouped, std::string *why)
{
    const Checker bad{why};
    int rc;
    if (c_dtype != GEMM_F32 && c_dtype != GEMM_BF16)
        return bad(GEMM_ERR_INVALID, "c_dtype must be GEMM_F32 or GEMM_BF16");
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxDim) return bad(GEMM_ERR_INVALID, "N and K must be in 0..2^31 - 1025");
    if (grouped) {
        if ((rc = check_groups(bad, groups, rows, offsets))) return rc;
    } else if (rows < 0 || rows > kMaxDim) {
        return bad(GEMM_ERR_INVALID, "M must be in 0..2^31 - 1025");
    }
    if (rows == 0 || N == 0) return GEMM_OK;
    if (groups * N > kMaxDim) return bad(GEMM_ERR_INVALID, "groups * N must be below 2^31 - 1024");
    if (too_many_tiles(rows, groups, N)) return bad(GEMM_ERR_INVALID, "the product has 2^31 tiles or more");
    if ((rc = check_c(bad, C, ldc, rows, N, c_dtype))) return rc;
    if (K == 0) return GEMM_OK;
    if ((rc = check_mx4_operand(bad, rows, K, ac, aq, as, al))) return rc;
    if ((rc = check_mx4_operand(bad, groups * N, K, bc, bq, bs, bl))) return rc;
    if (groups > 1 && N * bq >= (int64_t{1} << 40))
        return bad(GEMM_ERR_INVALID, "a group's matrix must span less than 2^40 bytes");
    return GEMM_OK;
}

int check_quantise(int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld, int64_t stride,
                   int src_dtype, const void *codes, int64_t ldq, const void *scales, int64_t lds, std::string *why)
{
    const Checker bad{why};
    if (layout != GEMM_B_ROW_MAJOR && layout != GEMM_B_COL_MAJOR)
        return bad(GEMM_ERR_INVALID, "layout must be GEMM_B_ROW_MAJOR or GEMM_B_COL_MAJOR");
    if (src_dtype != GEMM_F32 && src_dtype != GEMM_BF16)
        return bad(GEMM_ERR_INVALID, "src_dtype must be GEMM_F32 or GEMM_BF16");
    if (batch < 0 || rows < 0 || K < 0 || batch > kMaxDim || rows > kMaxDim || K > kMaxDim)
        return bad(GEMM_ERR_INVALID, "batch, rows and K must be in 0..2^31 - 1025");
    if (batch == 0 || rows == 0 || K == 0) return GEMM_OK;
    if (batch * rows > kMaxDim) return bad(GEMM_ERR_INVALID, "batch * rows must be below 2^31 - 1024");
    if (!src) return bad(GEMM_ERR_INVALID, "src is NULL");
    const bool k_rows = layout == GEMM_B_ROW_MAJOR;
    const int64_t src_rows = k_rows ? K : rows, src_cols = k_rows ? rows : K;
    if (ld < src_cols || ld > kMaxLd) return bad(GEMM_ERR_INVALID, "ld must be at least a row of src and at most 2^36");
    if (beyond_memory(src_rows, ld)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    if (batch > 1 && (stride < (src_rows - 1) * ld + src_cols || stride > kMaxStride))
        return bad(GEMM_ERR_INVALID, "stride must reach past a matrix and stay within 2^37");
    if (reinterpret_cast<uintptr_t>(src) % (src_dtype == GEMM_BF16 ? 2 : 4))
        return bad(GEMM_ERR_ALIGNMENT, "src is not aligned to its element size");
    return check_mx4_operand(bad, batch * rows, K, codes, ldq, scales, lds);
}

int check_dequantise(int64_t rows, int64_t K, const void *codes, int64_t ldq, const void *scales, int64_t lds,
                     const void *dst, int64_t ldd, int dst_dtype, std::string *why)
{
    const Checker bad{why};
    if (dst_dtype != GEMM_F32 && dst_dtype != GEMM_BF16)
        return bad(GEMM_ERR_INVALID, "dst_dtype must be GEMM_F32 or GEMM_BF16");
    if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim)
        return bad(GEMM_ERR_INVALID, "rows and K must be in 0..2^31 - 1025");
    if (rows == 0 || K == 0) return GEMM_OK;
    if (!dst) return bad(GEMM_ERR_INVALID, "dst is NULL");
    if (ldd < K || ldd > kMaxLd) return bad(GEMM_ERR_INVALID, "ldd must satisfy K <= ldd <= 2^36");
    if (beyond_memory(rows, ldd)) return bad(GEMM_ERR_INVALID, kBeyondMemory);
    if (reinterpret_cast<uintptr_t>(dst) % (dst_dtype == GEMM_BF16 ? 2 : 4))
        return bad(GEMM_ERR_ALIGNMENT, "dst is not aligned to its element size");
    return check_mx4_operand(bad, rows, K, codes, ldq, scales, lds);
}

// ------------------------------------------------------------- tensor maps

int encode(gemm_ctx *h, CUtensorMap *map, CUtensorMapDataType type, int rank, uintptr_t base, const int64_t *dims,
           const int64_t *strides, const int *box, CUtensorMapSwizzle swizzle, const char *what)
{
    cuuint64_t d[5], st[4];
    cuuint32_t b[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        b[i] = static_cast<cuuint32_t>(box[i]);
        es[i] = 1;
        if (i + 1 < rank) st[i] = static_cast<cuuint64_t>(strides[i]);
    }
    const CUresult r = dg::g_encode(map, type, static_cast<cuuint32_t>(rank), reinterpret_cast<void *>(base), d, st, b,
                                    es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GEMM_OK;
    char msg[128];
    std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (%d) for %s", static_cast<int>(r), what);
    return fail(h, GEMM_ERR_CUDA, msg);
}

CUtensorMapDataType float_type(int es)
{
    return es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}

// 128-byte rows of an MN-major operand; 32-bit elements need 32-byte atoms.
CUtensorMapSwizzle mn_swizzle(int es)
{
    return es == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_128B_ATOM_32B;
}

// `groups` matrices of rows x cols (pitch ld, group stride in elements), MN-major:
// cols is the MMA's M side.  Whole 128-byte column chunks take one box a stage
// ({column, row, chunk, group}), else one box a chunk ({column, row, group}).
int encode_mn(gemm_ctx *h, CUtensorMap *map, int es, const void *base, int64_t rows, int64_t cols, int64_t ld,
              int64_t groups, int64_t stride, int box_cols, bool chunks)
{
    const int chunk = 128 / es;
    if (chunks) {
        const int64_t dims[4] = {chunk, rows, cols / chunk, groups};
        const int64_t st[3] = {ld * es, chunk * es, (groups > 1 ? stride : ld) * es};
        const int box[4] = {chunk, chunk, box_cols / chunk, 1};
        return encode(h, map, float_type(es), 4, reinterpret_cast<uintptr_t>(base), dims, st, box, mn_swizzle(es),
                      "row-major B in column chunks");
    }
    const int64_t dims[3] = {cols, rows, groups};
    const int64_t st[2] = {ld * es, (groups > 1 ? stride : ld) * es};
    const int box[3] = {chunk, chunk, 1};
    return encode(h, map, float_type(es), 3, reinterpret_cast<uintptr_t>(base), dims, st, box, mn_swizzle(es),
                  "row-major B");
}

// The zero-extending view of a ragged contraction (ragged.cu): {column, y < BK,
// z, chunk}, y and z both stepping one row, so coordinates (y, z) are row
// y + z; a box at (n - BK, r) reads zeros, then rows r .. r + n - 1.  BK =
// 128 bytes / es rows.
int encode_ragged_k(gemm_ctx *h, CUtensorMap *map, int es, const void *base, int64_t rows, int64_t cols, int64_t ld,
                    int box_cols, bool chunks)
{
    const int chunk = 128 / es;  // also BK
    const uintptr_t b = reinterpret_cast<uintptr_t>(base);
    if (chunks) {
        const int64_t dims[4] = {chunk, chunk, rows, cols / chunk};
        const int64_t st[3] = {ld * es, ld * es, chunk * es};
        const int box[4] = {chunk, chunk, 1, box_cols / chunk};
        return encode(h, map, float_type(es), 4, b, dims, st, box, mn_swizzle(es),
                      "a ragged contraction's operand in column chunks");
    }
    const int64_t dims[3] = {cols, chunk, rows};
    const int64_t st[2] = {ld * es, ld * es};
    const int box[3] = {chunk, chunk, 1};
    return encode(h, map, float_type(es), 3, b, dims, st, box, mn_swizzle(es), "a ragged contraction's operand");
}

// K-major: {k, row, group}, boxes of one 128-byte K slice.
int encode_k_major(gemm_ctx *h, CUtensorMap *map, CUtensorMapDataType type, int es, const void *base, int64_t K,
                   int64_t rows, int64_t ld, int64_t groups, int64_t stride, int box_k, int box_rows,
                   CUtensorMapSwizzle swizzle, bool grouped, const char *what)
{
    const int64_t dims[3] = {K, rows, groups};
    const int64_t st[2] = {ld * es, (groups > 1 ? stride : ld) * es};
    const int box[3] = {box_k, box_rows, 1};
    return encode(h, map, type, grouped ? 3 : 2, reinterpret_cast<uintptr_t>(base), dims, st, box, swizzle, what);
}

// The handle's first grouped or 4-bit product prepares the kernels; the call
// may be captured, and loading them is no part of the graph.
int prepare(gemm_ctx *h)
{
    if (h->ragged_ready) return GEMM_OK;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) {
        e = dg::prepare_ragged();
        cudaThreadExchangeStreamCaptureMode(&mode);
    }
    if (e != cudaSuccess) return cuda_fail(h, e, "preparing the grouped kernels");
    h->ragged_ready = true;
    return GEMM_OK;
}

dg::RaggedTile tile_for(const gemm_ctx *h, int kind, bool ragged_k, int64_t rows, int64_t groups, int64_t P,
                        int64_t Q, int64_t K)
{
    if (h->ragged_tile) {
        dg::RaggedTile t;
        t.split = std::max(1, h->ragged_tile / 10000);
        t.ctas = h->ragged_tile / 1000 % 10;
        t.bn = h->ragged_tile % 1000;
        if (ragged_k) t.bn = t.bn == 224 ? 256 : std::max(t.bn, 128);  // whole 128-byte column chunks per CTA
        if (kind == dg::kRaggedMx4) t.bn = std::min(t.bn, 224);        // two accumulators beside the scales
        return t;
    }
    const int sms = h->max_ctas > 0 ? std::min(h->max_ctas, h->sm_count) : h->sm_count;
    return dg::ragged_pick_tile(kind, ragged_k, rows, static_cast<int>(groups), P, Q, K, sms, h->split_k == 0);
}

dg::RaggedArgs common_args(const gemm_ctx *h, const int64_t *offsets, int64_t groups, int64_t rows, int64_t P,
                           int64_t Q, int64_t K, void *C, int64_t ldc, int c_dtype, cudaStream_t stream)
{
    dg::RaggedArgs a;
    a.offsets = offsets;
    a.groups = static_cast<int>(groups);
    a.rows = static_cast<int>(rows);
    a.P = static_cast<int>(P);
    a.Q = static_cast<int>(Q);
    a.K = static_cast<int>(K);
    a.C = C;
    a.ldc = ldc;
    a.out_bf16 = c_dtype == GEMM_BF16 ? 1 : 0;
    a.status = h->d_status;
    a.timeout_ns = h->timeout_ns;
    a.debug_drop = h->debug_drop;
    a.stream = stream;
    return a;
}

// Formatted in place: these calls may take only microseconds.
void set_path(gemm_ctx *h, const char *op, int kind, const dg::RaggedTile &t, const char *rest, bool ra, bool rb)
{
    const char *k = kind == dg::kRaggedMx4 ? "mx4" : kind == dg::kRaggedTf32 ? "tf32" : "bf16";
    char split[16] = "", path[128];
    if (t.split > 1) std::snprintf(split, sizeof split, "+splitk%d", t.split);
    std::snprintf(path, sizeof path, "%s_%s%s%dx%d%s%s%s%s", op, k, t.ctas == 2 ? "_pair" : "_", 128 * t.ctas, t.bn,
                  rest, ra ? "+repackA" : "", rb ? "+repackB" : "", split);
    h->last_path = path;
}

// A row-major operand that TMA can address: itself, or its copy in the
// workspace at a 16-byte pitch.
struct Repack {
    bool needed = false;
    int64_t ld = 0;
    size_t bytes = 0;
};

Repack plan_repack(const gemm_ctx *h, const void *src, int64_t ld, int64_t groups, int64_t stride, int64_t rows,
                   int64_t cols, int es)
{
    Repack r;
    r.needed = h->force_repack || !dg::tma_ready(src, ld, es) || (groups > 1 && (stride * es) % 16 != 0);
    if (r.needed) {
        r.ld = round_up(cols, 16 / es);
        r.bytes = static_cast<size_t>(round_up(groups * rows * r.ld * es, 256));
    }
    return r;
}

// One matrix, or `groups` of them that follow one another, as a copy job.
// `offsets`: skip the matrices of groups without rows.
dg::RepackJob job_of(const Repack &r, uint8_t *dst, const void *src, int64_t ld, int64_t groups, int64_t rows,
                     int64_t cols, const int64_t *offsets)
{
    dg::RepackJob j;
    if (!r.needed) return j;
    j.src = src;
    j.lds = ld;
    j.dst = dst;
    j.ldd = r.ld;
    j.rows = groups * rows;
    j.cols = cols;
    j.offsets = reinterpret_cast<const long long *>(offsets);
    j.rows_per = rows;
    return j;
}

// Copies the operands that TMA cannot address into the workspace, A and B in
// one launch; B's matrices one launch each when they do not follow one another.
int run_repack(gemm_ctx *h, const Repack &ra, const void *A, int64_t lda, int64_t rows_a, int64_t cols_a,
               const Repack &rb, const void *B, int64_t ldb, int64_t groups, int64_t stride_b, int64_t rows_b,
               int64_t cols_b, const int64_t *offsets, int es, cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(h->ws);
    const bool flat = groups == 1 || stride_b == rows_b * ldb;
    const dg::RepackJob a = job_of(ra, ws, A, lda, 1, rows_a, cols_a, nullptr);
    for (int64_t g = 0; g < (rb.needed && !flat ? groups : 1); ++g) {
        const dg::RepackJob b =
            job_of(rb, ws + ra.bytes + g * rows_b * rb.ld * es, static_cast<const uint8_t *>(B) + g * stride_b * es, ldb,
                   flat ? groups : 1, rows_b, cols_b, offsets ? offsets + g : nullptr);
        const cudaError_t e = dg::launch_repack_jobs(g == 0 ? a : dg::RepackJob(), b, es, h->sm_count, stream);
        if (e != cudaSuccess) return cuda_fail(h, e, "repack launch");
        ++h->launches;
    }
    return GEMM_OK;
}

int run_mx4(gemm_ctx *h, int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets, const void *ac,
            int64_t aq, const void *as, int64_t al, const void *bc, int64_t bq, const void *bs, int64_t bl, void *C,
            int64_t ldc, int c_dtype, cudaStream_t stream)
{
    if (rows == 0 || N == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h->device);
    int rc = prepare(h);
    if (rc) return rc;
    const int kind = dg::kRaggedMx4;
    const dg::RaggedTile t = tile_for(h, kind, false, rows, groups, N, 0, K);
    dg::RaggedArgs a = common_args(h, offsets, groups, rows, N, 0, K, C, ldc, c_dtype, stream);
    alignas(64) CUtensorMap tmP = {}, tmQ = {};
    if (K > 0) {
        const int64_t Kp = round_up(K, GEMM_MX4_BLOCK);
        const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
        const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
        rc = encode_k_major(h, &tmP, u8, 1, bc, Kp / 2, N, bq, groups, N * bq, 128, dg::kRaggedP, sw, true,
                                "the codes of B");
        if (!rc) rc = encode_k_major(h, &tmQ, u8, 1, ac, Kp / 2, rows, aq, 1, 0, 128, t.bn / t.ctas, sw, false,
                                     "the codes of A");
        if (rc) return rc;
        a.scale_p = static_cast<const uint8_t *>(bs);
        a.lds_p = bl;
        a.scale_q = static_cast<const uint8_t *>(as);
        a.lds_q = al;
    }
    const cudaError_t e = dg::launch_ragged(kind, false, false, t, tmP, tmQ, a, h->sm_count, h->max_ctas);
    if (e != cudaSuccess) return cuda_fail(h, e, "4-bit product launch");
    ++h->launches;
    set_path(h, offsets ? "grouped" : "tc", kind, t, "", false, false);
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_grouped_validate(int layout_b, int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                          const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b, const void *C,
                          int64_t ldc, int dtype, int c_dtype)
{
    return check_grouped(layout_b, groups, rows, N, K, offsets, A, lda, B, ldb, stride_b, C, ldc, dtype, c_dtype,
                         nullptr);
}

int gemm_grouped_wgrad_validate(int64_t groups, int64_t rows, int64_t M, int64_t N, const int64_t *offsets,
                                const void *A, int64_t lda, const void *B, int64_t ldb, const void *C, int64_t ldc,
                                int64_t stride_c, int dtype, int c_dtype)
{
    take_nan_flag(c_dtype);
    return check_wgrad(groups, rows, M, N, offsets, A, lda, B, ldb, C, ldc, stride_c, dtype, c_dtype, nullptr);
}

int gemm_grouped_run(gemm_handle_t h, int layout_b, int64_t groups, int64_t rows, int64_t N, int64_t K,
                     const int64_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b,
                     void *C, int64_t ldc, int dtype, int c_dtype, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    int rc = check_grouped(layout_b, groups, rows, N, K, offsets, A, lda, B, ldb, stride_b, C, ldc, dtype, c_dtype,
                           &why);
    if (rc) return fail(h, rc, why);
    if (rows == 0 || N == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h->device);
    if ((rc = prepare(h))) return rc;
    const int es = dtype == GEMM_BF16 ? 2 : 4;
    const int kind = dtype == GEMM_BF16 ? dg::kRaggedBf16 : dg::kRaggedTf32;
    const bool row = layout_b == GEMM_B_ROW_MAJOR;
    const int64_t rows_b = row ? K : N, cols_b = row ? N : K;
    const dg::RaggedTile t = tile_for(h, kind, false, rows, groups, N, 0, K);
    dg::RaggedArgs a = common_args(h, offsets, groups, rows, N, 0, K, C, ldc, c_dtype, stream);
    alignas(64) CUtensorMap tmP = {}, tmQ = {};
    dg::WorkspaceUse ws(h, stream);
    Repack ra, rb;
    if (K > 0) {
        ra = plan_repack(h, A, lda, 1, 0, rows, K, es);
        rb = plan_repack(h, B, ldb, groups, stride_b, rows_b, cols_b, es);
        if (ra.needed || rb.needed) {
            if ((rc = ws.acquire(ra.bytes + rb.bytes))) return rc;
            if ((rc = run_repack(h, ra, A, lda, rows, K, rb, B, ldb, groups, stride_b, rows_b, cols_b, offsets, es, stream)))
                return rc;
        }
        if (ra.needed) {
            A = h->ws;
            lda = ra.ld;
        }
        if (rb.needed) {
            B = static_cast<uint8_t *>(h->ws) + ra.bytes;
            ldb = rb.ld;
            stride_b = rows_b * rb.ld;
        }
        a.p_chunks = row && N % (128 / es) == 0 ? 1 : 0;
        rc = row ? encode_mn(h, &tmP, es, B, K, N, ldb, groups, stride_b, dg::kRaggedP, a.p_chunks != 0)
                 : encode_k_major(h, &tmP, float_type(es), es, B, K, N, ldb, groups, stride_b, 128 / es, dg::kRaggedP,
                                  CU_TENSOR_MAP_SWIZZLE_128B, true, "column-major B");
        if (!rc)
            rc = encode_k_major(h, &tmQ, float_type(es), es, A, K, rows, lda, 1, 0, 128 / es, t.bn / t.ctas,
                                CU_TENSOR_MAP_SWIZZLE_128B, false, "A");
        if (rc) return rc;
    }
    const cudaError_t e = dg::launch_ragged(kind, false, row, t, tmP, tmQ, a, h->sm_count, h->max_ctas);
    if (e != cudaSuccess) return cuda_fail(h, e, "grouped product launch");
    ++h->launches;
    set_path(h, "grouped", kind, t, row ? "_rowB" : "_colB", ra.needed, rb.needed);
    return ws.done();
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int gemm_grouped_wgrad(gemm_handle_t h, int64_t groups, int64_t rows, int64_t M, int64_t N, const int64_t *offsets,
                       const void *A, int64_t lda, const void *B, int64_t ldb, void *C, int64_t ldc, int64_t stride_c,
                       int dtype, int c_dtype, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const bool nan_on_error = take_nan_flag(c_dtype);
    int rc = check_wgrad(groups, rows, M, N, offsets, A, lda, B, ldb, C, ldc, stride_c, dtype, c_dtype, &why);
    if (rc) return fail(h, rc, why);
    if (M == 0 || N == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h->device);
    if ((rc = prepare(h))) return rc;
    const int es = dtype == GEMM_BF16 ? 2 : 4;
    const int kind = dtype == GEMM_BF16 ? dg::kRaggedBf16 : dg::kRaggedTf32;
    const dg::RaggedTile t = tile_for(h, kind, true, rows, groups, N, M, 0);
    dg::RaggedArgs a = common_args(h, offsets, groups, rows, N, M, 0, C, ldc, c_dtype, stream);
    a.stride_c = groups > 1 ? stride_c : 0;
    alignas(64) CUtensorMap tmP = {}, tmQ = {};
    dg::WorkspaceUse ws(h, stream);
    Repack ra, rb;
    if (rows > 0) {
        ra = plan_repack(h, A, lda, 1, 0, rows, M, es);
        rb = plan_repack(h, B, ldb, 1, 0, rows, N, es);
        if (ra.needed || rb.needed) {
            if ((rc = ws.acquire(ra.bytes + rb.bytes))) return rc;
            if ((rc = run_repack(h, ra, A, lda, rows, M, rb, B, ldb, 1, 0, rows, N, nullptr, es, stream))) return rc;
        }
        if (ra.needed) {
            A = h->ws;
            lda = ra.ld;
        }
        if (rb.needed) {
            B = static_cast<uint8_t *>(h->ws) + ra.bytes;
            ldb = rb.ld;
        }
        a.p_chunks = N % (128 / es) == 0 ? 1 : 0;
        a.q_chunks = M % (128 / es) == 0 ? 1 : 0;
        rc = encode_ragged_k(h, &tmP, es, B, rows, N, ldb, dg::kRaggedP, a.p_chunks != 0);
        if (!rc) rc = encode_ragged_k(h, &tmQ, es, A, rows, M, lda, t.bn / t.ctas, a.q_chunks != 0);
        if (rc) return rc;
    }
    cudaError_t e = dg::launch_ragged(kind, true, true, t, tmP, tmQ, a, h->sm_count, h->max_ctas);
    if (e != cudaSuccess) return cuda_fail(h, e, "weight gradient launch");
    ++h->launches;
    if (nan_on_error) {
        if ((e = dg::launch_nan_on_error(a, h->sm_count)) != cudaSuccess) return cuda_fail(h, e, "NaN launch");
        ++h->launches;
    }
    set_path(h, "grouped", kind, t, "_wgrad", ra.needed, rb.needed);
    return ws.done();
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int64_t gemm_mx4_code_pitch(int64_t K) { return K <= 0 ? 0 : round_up(round_up(K, GEMM_MX4_BLOCK) / 2, 16); }

int64_t gemm_mx4_scale_pitch(int64_t K) { return K <= 0 ? 0 : round_up(round_up(K, GEMM_MX4_BLOCK) / 32, 16); }

int gemm_mx4_quantise_validate(int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                               int64_t stride, int src_dtype, const void *codes, int64_t ldq, const void *scales,
                               int64_t lds)
{
    return check_quantise(layout, batch, rows, K, src, ld, stride, src_dtype, codes, ldq, scales, lds, nullptr);
}

int gemm_mx4_dequantise_validate(int64_t rows, int64_t K, const void *codes, int64_t ldq, const void *scales,
                                 int64_t lds, const void *dst, int64_t ldd, int dst_dtype)
{
    return check_dequantise(rows, K, codes, ldq, scales, lds, dst, ldd, dst_dtype, nullptr);
}

int gemm_mx4_validate(int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets, const void *a_codes,
                      int64_t a_ldq, const void *a_scales, int64_t a_lds, const void *b_codes, int64_t b_ldq,
                      const void *b_scales, int64_t b_lds, const void *C, int64_t ldc, int c_dtype)
{
    return check_mx4(groups, rows, N, K, offsets, a_codes, a_ldq, a_scales, a_lds, b_codes, b_ldq, b_scales, b_lds, C,
                     ldc, c_dtype, !(groups == 1 && offsets == nullptr), nullptr);
}

int gemm_mx4_quantise(gemm_handle_t h, int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                      int64_t stride, int src_dtype, void *codes, int64_t ldq, void *scales, int64_t lds,
                      cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const int rc = check_quantise(layout, batch, rows, K, src, ld, stride, src_dtype, codes, ldq, scales, lds, &why);
    if (rc) return fail(h, rc, why);
    if (batch == 0 || rows == 0 || K == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h->device);
    const cudaError_t e = dg::launch_mx4_quantise(layout == GEMM_B_ROW_MAJOR, batch, rows, K, src, ld,
                                                  batch > 1 ? stride : 0, src_dtype == GEMM_BF16,
                                                  static_cast<uint8_t *>(codes), ldq, static_cast<uint8_t *>(scales),
                                                  lds, h->sm_count, stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "quantisation launch");
    ++h->launches;
    h->last_path = layout == GEMM_B_ROW_MAJOR ? "mx4_quantise_rowB" : "mx4_quantise_colB";
    return GEMM_OK;
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int gemm_mx4_dequantise(gemm_handle_t h, int64_t rows, int64_t K, const void *codes, int64_t ldq, const void *scales,
                        int64_t lds, void *dst, int64_t ldd, int dst_dtype, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const int rc = check_dequantise(rows, K, codes, ldq, scales, lds, dst, ldd, dst_dtype, &why);
    if (rc) return fail(h, rc, why);
    if (rows == 0 || K == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h->device);
    const cudaError_t e =
        dg::launch_mx4_dequantise(rows, K, static_cast<const uint8_t *>(codes), ldq,
                                  static_cast<const uint8_t *>(scales), lds, dst, ldd, dst_dtype == GEMM_BF16,
                                  h->sm_count, stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "dequantisation launch");
    ++h->launches;
    h->last_path = "mx4_dequantise";
    return GEMM_OK;
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int gemm_mx4_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *a_codes, int64_t a_ldq,
                 const void *a_scales, int64_t a_lds, const void *b_codes, int64_t b_ldq, const void *b_scales,
                 int64_t b_lds, void *C, int64_t ldc, int c_dtype, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const int rc = check_mx4(1, M, N, K, nullptr, a_codes, a_ldq, a_scales, a_lds, b_codes, b_ldq, b_scales, b_lds, C,
                             ldc, c_dtype, false, &why);
    if (rc) return fail(h, rc, why);
    return run_mx4(h, 1, M, N, K, nullptr, a_codes, a_ldq, a_scales, a_lds, b_codes, b_ldq, b_scales, b_lds, C, ldc,
                   c_dtype, stream);
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int gemm_mx4_grouped_run(gemm_handle_t h, int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                         const void *a_codes, int64_t a_ldq, const void *a_scales, int64_t a_lds, const void *b_codes,
                         int64_t b_ldq, const void *b_scales, int64_t b_lds, void *C, int64_t ldc, int c_dtype,
                         cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const int rc = check_mx4(groups, rows, N, K, offsets, a_codes, a_ldq, a_scales, a_lds, b_codes, b_ldq, b_scales,
                             b_lds, C, ldc, c_dtype, true, &why);
    if (rc) return fail(h, rc, why);
    return run_mx4(h, groups, rows, N, K, offsets, a_codes, a_ldq, a_scales, a_lds, b_codes, b_ldq, b_scales, b_lds, C,
                   ldc, c_dtype, stream);
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

}  // extern "C"
