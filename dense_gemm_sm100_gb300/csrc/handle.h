// The handle behind the C ABI and the helpers every entry point uses: error
// reporting, the stream-ordered workspace, TMA tensor-map encoding and the
// device guard.  Shared by the translation units that implement the C ABI.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <new>
#include <string>
#include <vector>

#include "../../include/gemm.h"

struct gemm_ctx {
    int device = 0;
    int sm_count = 0;
    int *d_status = nullptr;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    // Recorded on the caller's stream after every call that used the
    // workspace.  Calls on another stream wait on it, and growth does before
    // the old buffer is released (both in stream order).
    cudaEvent_t ws_event = nullptr;
    bool ws_event_recorded = false;
    unsigned long long ws_stream = 0;  // id of the stream it was recorded on
    // A call that used the present workspace was captured in a CUDA graph: the
    // graph may run at any later time, so growth keeps the buffer until the
    // handle goes.  So it does with a buffer that is outgrown during a capture,
    // which has no place in the graph for its release.
    bool ws_captured = false;
    std::vector<void *> ws_retired;
    std::string last_error;
    std::string last_path;
    int64_t launches = 0;
    int force_repack = 0;
    uint64_t timeout_ns = 4000000000ull;
    int simt_group_m = 0;
    int tc_group_m = 0;
    int max_ctas = 0;
    int simt_config = 0;  // 0: chosen per shape; else configuration index + 1
    int elementwise = 0;  // FP32 unaligned operands: element-wise producer (1) or re-pack (0)
    size_t ws_limit = 0;  // 0: none; else the workspace never grows beyond this many bytes
    int split_k = 0;      // 0: chosen per shape; 1: never; n > 1: n K slices (FP32 path)
    int stream_k = 0;     // FP32 tail: 0 chosen per shape, 1 slices, 2 stream-K
    int simt_small = 0;   // FP32 small-problem kernel: 0 chosen per shape, 1 never, 2 always
    int tc_cluster = 3;   // tensor-core mode: 1 one CTA per tile, 3 pair MMA
    int tc_tma_store = 1; // tensor-core epilogue writes C with TMA stores when C allows it
    int tc_slices = 0;    // pair MMA: K slices per ring stage (0: library's choice)
    bool ragged_ready = false;  // prepare_ragged has run for this handle
    int ragged_tile = 0;  // grouped and 4-bit products: 0 chosen, else 10000 * split + 1000 * CTAs + rows of a tile
    int debug_drop = 0;   // test hook (GEMM_OPT_DEBUG_DROP_LOAD)
    // gemm_run_host pipeline: copy streams and events (created on first use)
    cudaStream_t copy_in = nullptr, copy_out = nullptr;
    cudaEvent_t ev_start = nullptr, ev_done = nullptr;
    cudaEvent_t ev_a[16] = {}, ev_b[8] = {}, ev_c[16 * 8] = {};  // row panels, column panels, blocks
};

namespace dg {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;  // kernels index tiles with int
constexpr int64_t kMaxLd = int64_t{1} << 36;

// cuTensorMapEncodeTiled, looked up once by gemm_create.
extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

inline int fail(gemm_ctx *h, int code, const std::string &msg)
{
    if (h) h->last_error = msg;
    return code;
}

inline int cuda_fail(gemm_ctx *h, cudaError_t e, const char *what)
{
    cudaGetLastError();  // clear a non-sticky error so the next call starts clean
    return fail(h, GEMM_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

inline bool tma_ready(const void *p, int64_t ld, int es)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0;
}

// The end of the work queued on `stream` so far is what the workspace's next
// user waits for.
inline cudaError_t record_workspace_event(gemm_ctx *h, cudaStream_t stream)
{
    unsigned long long id = 0;
    cudaError_t e = cudaStreamGetId(stream, &id);
    if (e == cudaSuccess) e = cudaEventRecord(h->ws_event, stream);
    if (e == cudaSuccess) {
        h->ws_stream = id;
        h->ws_event_recorded = true;
    }
    return e;
}

// Before a call's first use of a workspace that is large enough: calls on
// different streams take turns.  (A capture cannot wait for work outside its
// graph; its launches are the caller's to order.)
inline int order_workspace(gemm_ctx *h, cudaStream_t stream)
{
    if (!h->ws_event_recorded) return GEMM_OK;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &capture);
    if (e == cudaSuccess && capture != cudaStreamCaptureStatusNone) return GEMM_OK;
    unsigned long long id = 0;  // not to be had from a stream that is being captured
    if (e == cudaSuccess) e = cudaStreamGetId(stream, &id);
    if (e == cudaSuccess && id != h->ws_stream) e = cudaStreamWaitEvent(stream, h->ws_event, 0);
    return e == cudaSuccess ? GEMM_OK : cuda_fail(h, e, "ordering the workspace's uses");
}

// Makes `need` bytes of workspace usable on `stream`.
//
// Growth is in stream order: the stream first waits for the last call that
// used the old buffer, then frees it and allocates the new one from the
// device's stream-ordered pool.  Nothing waits on the host, and work the caller
// queued on other streams is not held up.  While `stream` is being captured the
// new buffer is allocated outside the graph (memory that a graph's node
// allocates is there only while the graph runs, and later calls on the handle
// would use its address all the same).
inline int ensure_workspace(gemm_ctx *h, size_t need, cudaStream_t stream)
{
    if (need <= h->ws_bytes) return order_workspace(h, stream);
    if (h->ws_limit > 0 && need > h->ws_limit) {
        char msg[160];
        std::snprintf(msg, sizeof msg, "workspace of %zu bytes needed, limit %zu (GEMM_OPT_WORKSPACE_LIMIT)", need,
                      h->ws_limit);
        return fail(h, GEMM_ERR_NOMEM, msg);
    }
    size_t grow = h->ws_bytes + h->ws_bytes / 2;
    size_t bytes = need > grow ? need : grow;
    bytes = (bytes + (size_t{2} << 20) - 1) & ~((size_t{2} << 20) - 1);
    if (h->ws_limit > 0 && bytes > h->ws_limit) bytes = need;  // stay within the limit
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &capture);
    if (e != cudaSuccess) return cuda_fail(h, e, "growth of the workspace");
    const bool capturing = capture != cudaStreamCaptureStatusNone;
    if (h->ws && (capturing || h->ws_captured)) {
        try {
            h->ws_retired.push_back(h->ws);
        } catch (const std::bad_alloc &) {
            return GEMM_ERR_NOMEM;
        }
    } else if (h->ws) {
        // Earlier calls (on this or another stream) may still read the old buffer.
        if (h->ws_event_recorded) e = cudaStreamWaitEvent(stream, h->ws_event, 0);
        if (e == cudaSuccess) e = cudaFreeAsync(h->ws, stream);
        if (e != cudaSuccess) return cuda_fail(h, e, "stream-ordered release of the old workspace");
    }
    h->ws = nullptr;
    h->ws_bytes = 0;
    h->ws_event_recorded = false;
    h->ws_captured = capturing;
    if (capturing) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // of this thread, for the one call
        e = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e == cudaSuccess) {
            e = cudaMalloc(&h->ws, bytes);
            cudaThreadExchangeStreamCaptureMode(&mode);
        }
    } else {
        e = cudaMallocAsync(&h->ws, bytes, stream);
    }
    if (e != cudaSuccess) {
        h->ws = nullptr;
        h->ws_captured = false;
        cudaGetLastError();
        return fail(h, GEMM_ERR_NOMEM, std::string("workspace allocation: ") + cudaGetErrorString(e));
    }
    h->ws_bytes = bytes;
    // cudaMalloc's memory is there for every stream at once
    if (!capturing && (e = record_workspace_event(h, stream)) != cudaSuccess)
        return cuda_fail(h, e, "workspace-use event");
    return GEMM_OK;
}

// After a call whose launches read or write the workspace.
inline int note_workspace_use(gemm_ctx *h, cudaStream_t stream)
{
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &capture);
    if (e == cudaSuccess && capture == cudaStreamCaptureStatusActive) {
        // an event recorded into the graph could not be waited for outside it
        h->ws_captured = true;
        return GEMM_OK;
    }
    if (e == cudaSuccess) e = record_workspace_event(h, stream);
    return e == cudaSuccess ? GEMM_OK : cuda_fail(h, e, "workspace-use event");
}

// One call's use of the workspace.  Its end is recorded however the call
// leaves: a launch that fails, or an exception, may follow launches that
// already work on the buffer.
class WorkspaceUse {
  public:
    WorkspaceUse(gemm_ctx *h, cudaStream_t stream) : h_(h), stream_(stream) {}
    ~WorkspaceUse()
    {
        try {
            done();
        } catch (...) {
        }
    }
    WorkspaceUse(const WorkspaceUse &) = delete;
    WorkspaceUse &operator=(const WorkspaceUse &) = delete;

    int acquire(size_t need)
    {
        const int rc = ensure_workspace(h_, need, stream_);
        held_ = rc == GEMM_OK;
        return rc;
    }

    int done()
    {
        if (!held_) return GEMM_OK;
        held_ = false;
        return note_workspace_use(h_, stream_);
    }

  private:
    gemm_ctx *h_;
    cudaStream_t stream_;
    bool held_ = false;
};

inline int encode_2d(gemm_ctx *h, CUtensorMap *map, int es, const void *base, int64_t inner,
              int64_t outer, int64_t ld, int box_inner, int box_outer,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType dt = es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUresult r = g_encode(map, dt, 2, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char msg[160];
        std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (%d) for a %lld x %lld operand",
                      static_cast<int>(r), static_cast<long long>(outer), static_cast<long long>(inner));
        return fail(h, GEMM_ERR_CUDA, msg);
    }
    return GEMM_OK;
}

class DeviceGuard {
  public:
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        if (prev_ != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev_) cudaSetDevice(prev_);
    }

  private:
    int prev_ = -1;
};

}  // namespace dg
