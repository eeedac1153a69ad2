// Launch interface of the orthogonalised update (ortho.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dg {

// Buffers of a group of matrices in the workspace.  m <= n are the matrix's
// sides, ldm and ldn rows of m and n elements rounded up to whole 128 bytes.
// Two-term numbers: plane 0 the FP16 value, plane 1 the rest.
struct OrthoBuffers {
    int m = 0, n = 0, ldm = 0, ldn = 0, batch = 0;
    uint8_t *x[2][2] = {};  // [this step's, the next one's][plane]: batch x m x ldn FP16
    uint8_t *a[2] = {};     // [plane]: batch x m x ldm FP16, zero diagonals
    uint8_t *b[2] = {};
    float *da = nullptr, *db = nullptr;  // diagonals: batch x ldm
    double *parts = nullptr;             // batch x ORTHO_PARTS sums of squares
    float *factors = nullptr;            // batch x ORTHO_FACTORS
};
constexpr int ORTHO_PARTS = 64, ORTHO_FACTORS = 7;

size_t ortho_bytes(int64_t m, int64_t n, bool split);  // of one matrix
void ortho_layout(OrthoBuffers &o, uint8_t *base, bool split);

// What the caller's matrices look like.
struct OrthoMatrices {
    const void *g = nullptr;
    long long ldg = 0, stride_g = 0;
    void *o = nullptr;
    long long ldo = 0, stride_o = 0;
    int rows = 0, cols = 0;
    bool bf16 = false;
    float eps = 0;
};

cudaError_t prepare_ortho();  // kernel attributes on the current device
// X = G / (|G| + eps), up to the factors; *launches counts kernels.
cudaError_t launch_ortho_start(const OrthoBuffers &w, const OrthoMatrices &u, bool split, int max_ctas,
                               cudaStream_t stream, int *launches);

enum OrthoStep : int { kOrthoA = 0, kOrthoB = 1, kOrthoX = 2 };

struct OrthoTile {
    int ctas = 1, bn = 128;
};
OrthoTile ortho_pick_tile(int step, bool split, int64_t batch, int64_t m, int64_t n, int sm_count);

struct OrthoProduct {
    int step = kOrthoA;
    bool split = false, first = false, last = false;
    int from = 0;  // X's buffer that is read; X is written to the other
    float ca = 0, cb = 0, cc = 0;
    OrthoTile tile;
    int *status = nullptr;
    uint64_t timeout_ns = 0;
    int debug_drop = 0;
    cudaStream_t stream = nullptr;
};
// Maps: P's planes, then Q's.
cudaError_t launch_ortho_product(const OrthoBuffers &w, const OrthoMatrices &u, const OrthoProduct &p,
                                 const CUtensorMap (&maps)[4], int sm_count, int max_ctas);

}  // namespace dg
