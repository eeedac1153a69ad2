// Launch interface of the grouped tensor-core kernel (ragged.cu) and of the
// microscaled 4-bit conversion kernels (mx4.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace dg {

// Operand kinds of the grouped kernel.
enum RaggedKind : int { kRaggedBf16 = 0, kRaggedTf32 = 1, kRaggedMx4 = 2 };

// The kernel computes, for every group g, D[p][q] = sum_k P_g[p][k] Q_g[q][k]
// and stores D[p][q] at C[row(q) * ldc + p]: P is the operand whose index runs
// along a row of C, so that a warp's 32 tensor-memory lanes write 32
// neighbouring elements of one row.
//   ragged rows (ragged_k = false): Q is A (rows x K, groups are row ranges),
//     P is B_g (K-major or MN-major), row(q) the row of A;
//   ragged K (ragged_k = true): P_g = B_g^T and Q_g = A_g^T, both MN-major
//     with the group's rows as K, row(q) = g's first row in C plus q.
struct RaggedArgs {
    const int64_t *offsets = nullptr;  // groups + 1 values on the device; null: one group of all rows
    int groups = 1;
    int rows = 0;         // rows of the ragged operands
    int P = 0;            // columns of C
    int Q = 0;            // ragged_k: rows of each group's C
    int K = 0;            // ragged rows: contraction length
    void *C = nullptr;
    int64_t ldc = 0;
    int64_t stride_c = 0;  // ragged_k: elements from one group's C to the next
    int out_bf16 = 0;
    int p_chunks = 0;  // MN-major P: tmP is the view in 128-byte column chunks
    int q_chunks = 0;  // the same for Q (ragged_k)
    // kRaggedMx4: scale bytes of B (rows of P, groups one after another) and A
    const uint8_t *scale_p = nullptr, *scale_q = nullptr;
    int64_t lds_p = 0, lds_q = 0;
    int *status = nullptr;
    uint64_t timeout_ns = 0;
    int debug_drop = 0;
    cudaStream_t stream = nullptr;
};

// Tile of a launch: `ctas` (1, or 2 for a pair) x 128 columns of C by bn rows,
// its contraction cut over `split` CTAs (ctas = 1 and bn <= 128 only).
struct RaggedTile {
    int ctas = 1;
    int bn = 0;
    int split = 1;
};

// Status word of a launch whose offsets decrease or leave [0, rows].
constexpr int kStatusBadOffsets = 0x200;

constexpr int kRaggedMaxGroups = 4096;
constexpr int kRaggedP = 128;    // rows of P one CTA stages
constexpr int kRaggedBlock = 32;  // elements that share a 4-bit scale

bool ragged_tile_ok(int split, int ctas, int bn);  // split 0: none
RaggedTile ragged_pick_tile(int kind, bool ragged_k, int64_t rows, int groups, int64_t P, int64_t Q, int64_t K,
                            int sm_count, bool may_split);

// K elements of one ring stage (128 bytes of a K-major row).
inline int ragged_bk(int kind) { return kind == kRaggedMx4 ? 256 : kind == kRaggedTf32 ? 32 : 64; }

// Sets the kernels' attributes on the current device: once per handle, before
// its first product (1.5 ms for the first handle of a process, whose creation
// it would hold up for callers who never use these kernels).
cudaError_t prepare_ragged();
// tmP / tmQ: the operand views of ragged_api.cu.
cudaError_t launch_ragged(int kind, bool ragged_k, bool p_mn, const RaggedTile &t, const CUtensorMap &tmP,
                          const CUtensorMap &tmQ, const RaggedArgs &a, int sm_count, int max_ctas);

// Behind a weight gradient (its arguments `a`): NaN to all of C where the
// offsets were refused or the status word holds an expired wait.
cudaError_t launch_nan_on_error(const RaggedArgs &a, int sm_count);

// Quantises `batch` matrices of `rows` x K elements (BF16 or FP32) to E2M1
// codes and E8M0 scales, batch * rows output rows.  k_rows: element (r, k) is
// src[k * ld + r] instead of src[r * ld + k].
cudaError_t launch_mx4_quantise(bool k_rows, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                                int64_t stride, bool src_bf16, uint8_t *codes, int64_t ldq, uint8_t *scales,
                                int64_t lds, int sm_count, cudaStream_t stream);
cudaError_t launch_mx4_dequantise(int64_t rows, int64_t K, const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                                  int64_t lds, void *dst, int64_t ldd, bool dst_bf16, int sm_count,
                                  cudaStream_t stream);

}  // namespace dg
