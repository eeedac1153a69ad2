// The C ABI of include/gemm_ortho.h: argument checks, the workspace's layout,
// tensor maps and the sequence of launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/gemm.h"
#include "../../include/gemm_ortho.h"
#include "handle.h"
#include "ortho.h"

using dg::cuda_fail;
using dg::fail;
using dg::kMaxLd;

namespace {

constexpr int64_t kMaxSide = int64_t{1} << 20;
constexpr size_t kGroupBytes = size_t{4} << 30;  // workspace of the matrices worked on at a time

int check(int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg, int64_t stride_g, const void *O,
          int64_t ldo, int64_t stride_o, int dtype, int steps, const float *coefficients, float eps, std::string *why)
{
    const auto bad = [&](int code, const char *msg) {
        if (why) *why = msg;
        return code;
    };
    if (dtype != GEMM_F32 && dtype != GEMM_BF16) return bad(GEMM_ERR_INVALID, "dtype must be GEMM_F32 or GEMM_BF16");
    if (steps < 1 || steps > GEMM_ORTHO_MAX_STEPS) return bad(GEMM_ERR_INVALID, "steps must be in 1..32");
    if (!coefficients) return bad(GEMM_ERR_INVALID, "coefficients is NULL");
    for (int i = 0; i < 3 * steps; ++i)
        if (!std::isfinite(coefficients[i])) return bad(GEMM_ERR_INVALID, "coefficients must be finite");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return bad(GEMM_ERR_INVALID, "eps must be finite and not negative");
    if (batch < 0 || batch > dg::kMaxDim) return bad(GEMM_ERR_INVALID, "batch must be in 0..2^31 - 1025");
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return bad(GEMM_ERR_INVALID, "rows and cols must be in 0..2^20");
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_OK;
    if (!G || !O) return bad(GEMM_ERR_INVALID, "G or O is NULL");
    if (ldg < cols || ldg > kMaxLd || ldo < cols || ldo > kMaxLd)
        return bad(GEMM_ERR_INVALID, "ldg and ldo must be at least cols and at most 2^36");
    if (ldg > (int64_t{1} << 44) / rows || ldo > (int64_t{1} << 44) / rows)
        return bad(GEMM_ERR_INVALID, "rows times pitch must stay within 2^44");
    if (batch > 1)
        for (const auto &[stride, ld] : {std::pair<int64_t, int64_t>(stride_g, ldg), {stride_o, ldo}})
            if (stride < (rows - 1) * ld + cols || stride > (int64_t{1} << 44) / batch)
                return bad(GEMM_ERR_INVALID, "strides must reach past a matrix, batch times stride stay within 2^44");
    const uintptr_t es = dtype == GEMM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(G) % es || reinterpret_cast<uintptr_t>(O) % es)
        return bad(GEMM_ERR_ALIGNMENT, "G or O is not aligned to its element size");
    return GEMM_OK;
}

constexpr CUtensorMapDataType kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;

// Rows of `k` elements along K, box_rows of them a box.
int encode_k(gemm_ctx *h, CUtensorMap *map, const void *base, int64_t k, int64_t ld, const dg::OrthoBuffers &w,
             int box_rows)
{
    const int64_t dims[3] = {k, w.m, w.batch}, strides[2] = {ld * 2, w.m * ld * 2};
    const int box[3] = {64, box_rows, 1};
    return dg::encode(h, map, kF16, 3, reinterpret_cast<uintptr_t>(base), dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, "an orthogonalisation's operand");
}

// X with its rows as K, in chunks of 64 columns.
int encode_x(gemm_ctx *h, CUtensorMap *map, const void *base, const dg::OrthoBuffers &w, int chunks)
{
    const int64_t dims[4] = {64, w.m, w.ldn / 64, w.batch};
    const int64_t strides[3] = {int64_t{w.ldn} * 2, 128, int64_t{w.m} * w.ldn * 2};
    const int box[4] = {64, 64, chunks, 1};
    return dg::encode(h, map, kF16, 4, reinterpret_cast<uintptr_t>(base), dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, "an orthogonalisation's X");
}

// `w.batch` matrices: the whole sequence.
int run_group(gemm_ctx *h, const dg::OrthoBuffers &w, const dg::OrthoMatrices &u, int steps, const float *coefficients,
              cudaStream_t stream)
{
    const bool split = !u.bf16;
    const int sms = h->max_ctas > 0 ? std::min(h->max_ctas, h->sm_count) : h->sm_count;
    int launches = 0;
    cudaError_t e = dg::launch_ortho_start(w, u, split, h->max_ctas, stream, &launches);
    h->launches += launches;
    if (e != cudaSuccess) return cuda_fail(h, e, "orthogonalisation launch");
    dg::OrthoProduct r;
    r.split = split;
    r.status = h->d_status;
    r.timeout_ns = h->timeout_ns;
    r.debug_drop = h->debug_drop;
    r.stream = stream;
    // [product][X's buffer that is read]
    alignas(64) CUtensorMap maps[3][2][4] = {};
    dg::OrthoTile tiles[3];
    for (int step : {dg::kOrthoA, dg::kOrthoB, dg::kOrthoX}) {
        if (h->ortho_tile) {
            tiles[step].ctas = h->ortho_tile / 1000;
            tiles[step].bn = h->ortho_tile % 1000;
            if (step != dg::kOrthoX) tiles[step].bn = std::min(tiles[step].bn, 128 * tiles[step].ctas);
            if (step == dg::kOrthoX) tiles[step].bn = std::max(tiles[step].bn, 64 * tiles[step].ctas);
        } else {
            tiles[step] = dg::ortho_pick_tile(step, split, w.batch, w.m, w.n, sms);
        }
        const int q_rows = tiles[step].bn / tiles[step].ctas;
        for (int from = 0; from < 2; ++from)
            for (int pl = 0; pl < (split ? 2 : 1); ++pl) {
                CUtensorMap *p = &maps[step][from][pl], *q = &maps[step][from][2 + pl];
                int rc = GEMM_OK;
                if (step == dg::kOrthoA) {
                    rc = encode_k(h, p, w.x[from][pl], w.n, w.ldn, w, 128);
                    if (!rc) rc = encode_k(h, q, w.x[from][pl], w.n, w.ldn, w, q_rows);
                } else if (step == dg::kOrthoB && from == 0) {  // the same for both
                    rc = encode_k(h, p, w.a[pl], w.m, w.ldm, w, 128);
                    if (!rc) rc = encode_k(h, q, w.a[pl], w.m, w.ldm, w, q_rows);
                } else if (step == dg::kOrthoX) {
                    if (from == 0) rc = encode_k(h, p, w.b[pl], w.m, w.ldm, w, 128);
                    if (from == 1) *p = maps[step][0][pl];
                    if (!rc) rc = encode_x(h, q, w.x[from][pl], w, q_rows / 64);
                }
                if (rc) return rc;
            }
    }
    for (int k = 0; k < steps; ++k) {
        r.first = k == 0;
        r.last = k == steps - 1;
        r.from = k & 1;
        r.ca = coefficients[3 * k];
        r.cb = coefficients[3 * k + 1];
        r.cc = coefficients[3 * k + 2];
        for (int step : {dg::kOrthoA, dg::kOrthoB, dg::kOrthoX}) {
            r.step = step;
            r.tile = tiles[step];
            e = dg::launch_ortho_product(w, u, r, maps[step][step == dg::kOrthoB ? 0 : r.from], h->sm_count,
                                         h->max_ctas);
            if (e != cudaSuccess) return cuda_fail(h, e, "orthogonalisation launch");
            ++h->launches;
        }
    }
    char path[128];
    std::snprintf(path, sizeof path, "ortho_%s_%dx%d_%dx%d_%dx%d%s", split ? "f16x2" : "f16", 128 * tiles[0].ctas,
                  tiles[0].bn, 128 * tiles[1].ctas, tiles[1].bn, 128 * tiles[2].ctas, tiles[2].bn,
                  u.rows > u.cols ? "_turned" : "");
    h->last_path = path;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_orthogonalise_validate(int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg,
                                int64_t stride_g, const void *O, int64_t ldo, int64_t stride_o, int dtype, int steps,
                                const float *coefficients, float eps)
{
    return check(batch, rows, cols, G, ldg, stride_g, O, ldo, stride_o, dtype, steps, coefficients, eps, nullptr);
}

int gemm_orthogonalise(gemm_handle_t h, int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg,
                       int64_t stride_g, void *O, int64_t ldo, int64_t stride_o, int dtype, int steps,
                       const float *coefficients, float eps, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    int rc = check(batch, rows, cols, G, ldg, stride_g, O, ldo, stride_o, dtype, steps, coefficients, eps, &why);
    if (rc) return fail(h, rc, why);
    if (batch == 0 || rows == 0 || cols == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h);
    cudaError_t e = dg::prepare_ortho();
    if (e != cudaSuccess) return cuda_fail(h, e, "preparing the orthogonalisation's kernels");
    const bool split = dtype == GEMM_F32;
    dg::OrthoBuffers w;
    w.m = static_cast<int>(std::min(rows, cols));
    w.n = static_cast<int>(std::max(rows, cols));
    w.ldm = static_cast<int>(dg::round_up(w.m, 64));
    w.ldn = static_cast<int>(dg::round_up(w.n, 64));
    const size_t each = dg::ortho_bytes(w.m, w.n, split), slack = 16 * 256;
    size_t room = kGroupBytes;
    if (h->ws_limit > 0 && h->ws_limit < room) room = h->ws_limit;
    const int64_t group = std::max<int64_t>(1, std::min<int64_t>({batch, room > slack ? int64_t((room - slack) / each) : 1,
                                                                 int64_t{1} << 20}));
    dg::WorkspaceUse ws(h, stream);
    if ((rc = ws.acquire(static_cast<size_t>(group) * each + slack))) return rc;
    dg::OrthoMatrices u;
    u.ldg = ldg;
    u.stride_g = batch > 1 ? stride_g : 0;
    u.ldo = ldo;
    u.stride_o = batch > 1 ? stride_o : 0;
    u.rows = static_cast<int>(rows);
    u.cols = static_cast<int>(cols);
    u.bf16 = dtype == GEMM_BF16;
    u.eps = eps;
    const int64_t es = u.bf16 ? 2 : 4;
    for (int64_t b = 0; b < batch; b += group) {
        w.batch = static_cast<int>(std::min(group, batch - b));
        dg::ortho_layout(w, static_cast<uint8_t *>(h->ws), split);
        u.g = static_cast<const uint8_t *>(G) + b * u.stride_g * es;
        u.o = static_cast<uint8_t *>(O) + b * u.stride_o * es;
        if ((rc = run_group(h, w, u, steps, coefficients, stream))) return rc;
    }
    return ws.done();
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

}  // extern "C"
