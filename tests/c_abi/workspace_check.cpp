// The handle's workspace (csrc/handle.h) against a model of the CUDA runtime,
// on the CPU: the few runtime calls that it makes are defined here and keep a
// record, so that the order of allocations, releases, events and captures can
// be checked without a GPU.  Usage: workspace_check <scenario>; exit code 0
// when every check holds.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <vector>

#include "handle.h"

PFN_cuTensorMapEncodeTiled_v12000 dg::g_encode = nullptr;

namespace {

struct Stream {
    bool capturing = false;
};

std::vector<std::string> calls;          // what the code under test asked for
std::set<void *> async_blocks, blocks;   // live memory by allocator
cudaStreamCaptureMode mode = cudaStreamCaptureModeGlobal;
bool refuse_memory = false;
int checks_failed = 0;

Stream *of(cudaStream_t s) { return reinterpret_cast<Stream *>(s); }
cudaStream_t handle_of(Stream &s) { return reinterpret_cast<cudaStream_t>(&s); }

void check(bool ok, const char *what)
{
    if (ok) return;
    std::printf("failed: %s\n", what);
    ++checks_failed;
}

int count(const char *name)
{
    int n = 0;
    for (const std::string &c : calls) n += c.compare(0, std::strlen(name), name) == 0 ? 1 : 0;
    return n;
}

}  // namespace

extern "C" {

cudaError_t cudaGetLastError(void) { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "an error of the model"; }

cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus *out)
{
    *out = of(s)->capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}

cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long *id)
{
    if (of(s)->capturing) return cudaErrorStreamCaptureUnsupported;
    *id = reinterpret_cast<uintptr_t>(s);
    return cudaSuccess;
}

cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *m)
{
    const cudaStreamCaptureMode old = mode;
    mode = *m;
    *m = old;
    return cudaSuccess;
}

// On a capturing stream these two become nodes of the graph.
cudaError_t cudaMallocAsync(void **p, size_t bytes, cudaStream_t s)
{
    calls.push_back(of(s)->capturing ? "malloc node" : "mallocAsync");
    if (refuse_memory) return cudaErrorMemoryAllocation;
    *p = std::malloc(bytes < 64 ? bytes : 64);
    async_blocks.insert(*p);
    return cudaSuccess;
}

cudaError_t cudaFreeAsync(void *p, cudaStream_t s)
{
    calls.push_back(of(s)->capturing ? "free node" : "freeAsync");
    check(async_blocks.erase(p) == 1, "cudaFreeAsync got a block of cudaMallocAsync");
    return cudaSuccess;
}

// Unsafe while any stream captures in the global mode of the thread.
cudaError_t cudaMalloc(void **p, size_t bytes)
{
    calls.push_back("malloc");
    if (mode != cudaStreamCaptureModeRelaxed) return cudaErrorStreamCaptureUnsupported;
    if (refuse_memory) return cudaErrorMemoryAllocation;
    *p = std::malloc(bytes < 64 ? bytes : 64);
    blocks.insert(*p);
    return cudaSuccess;
}

cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t s)
{
    calls.push_back(of(s)->capturing ? "record node" : "record");
    return cudaSuccess;
}

// An event recorded outside a capture cannot be waited for inside it.
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t, unsigned int)
{
    calls.push_back("wait");
    return of(s)->capturing ? cudaErrorStreamCaptureIsolation : cudaSuccess;
}

}  // extern "C"

namespace {

constexpr size_t MB = size_t{1} << 20;

int use(gemm_ctx *h, size_t bytes, Stream &s)
{
    const int rc = dg::ensure_workspace(h, bytes, handle_of(s));
    return rc ? rc : dg::note_workspace_use(h, handle_of(s));
}

// The first call that needs the workspace is captured.
void growth_in_capture()
{
    gemm_ctx h;
    Stream s;
    s.capturing = true;
    check(use(&h, MB, s) == GEMM_OK, "the captured call succeeds");
    check(count("malloc node") == 0, "its memory does not belong to the graph");
    check(h.ws != nullptr && blocks.count(h.ws) == 1 && h.ws_bytes >= MB, "it is the handle's");
    check(mode == cudaStreamCaptureModeGlobal, "the thread's capture mode is as it was");
    void *first = h.ws;
    s.capturing = false;
    check(use(&h, MB, s) == GEMM_OK && h.ws == first, "an eager call that fits uses the same memory");
    check(use(&h, 64 * MB, s) == GEMM_OK && h.ws != first, "an eager call that does not fit gets new memory");
    check(blocks.count(first) == 1 && count("freeAsync") == 0, "the graph keeps what it was captured with");
}

// The workspace was used eagerly and grows while a later call is captured.
void eager_then_growth_in_capture()
{
    gemm_ctx h;
    Stream s;
    check(use(&h, MB, s) == GEMM_OK, "the eager call succeeds");
    void *first = h.ws;
    calls.clear();
    s.capturing = true;
    check(use(&h, 64 * MB, s) == GEMM_OK && h.ws != first, "the captured call grows the workspace");
    check(count("wait") == 0 && count("free") == 0 && count("malloc node") == 0, "and nothing of that enters the graph");
    check(async_blocks.count(first) == 1, "the old memory, perhaps still in use, stays");
    s.capturing = false;
    check(use(&h, 256 * MB, s) == GEMM_OK, "the next eager growth succeeds");
}

void no_memory_in_capture()
{
    gemm_ctx h;
    Stream s;
    s.capturing = true;
    refuse_memory = true;
    check(use(&h, MB, s) == GEMM_ERR_NOMEM, "the captured call reports it");
    check(h.ws == nullptr && h.ws_bytes == 0 && mode == cudaStreamCaptureModeGlobal, "the handle is as it was");
    refuse_memory = false;
    s.capturing = false;
    check(use(&h, MB, s) == GEMM_OK && async_blocks.count(h.ws) == 1, "and usable");
}

// Calls on two streams that the caller does not order share the workspace.
void two_streams()
{
    gemm_ctx h;
    Stream a, b;
    check(use(&h, MB, a) == GEMM_OK, "a call on the first stream");
    calls.clear();
    check(use(&h, MB, a) == GEMM_OK && count("wait") == 0, "calls on one stream are in order by themselves");
    calls.clear();
    check(use(&h, MB, b) == GEMM_OK && count("wait") == 1, "a call on another stream waits for the last use");
    check(calls.front() == "wait", "before it touches the workspace");
    calls.clear();
    check(use(&h, MB, a) == GEMM_OK && count("wait") == 1, "and back");
    a.capturing = b.capturing = true;
    calls.clear();
    check(use(&h, MB, b) == GEMM_OK && count("wait") == 0, "a capture cannot wait for work outside the graph");
}

// Nothing but the allocation itself happened on the stream that grew the
// workspace (the call failed after it).
void allocated_on_another_stream()
{
    gemm_ctx h;
    Stream a, b;
    check(dg::ensure_workspace(&h, MB, handle_of(a)) == GEMM_OK, "growth on the first stream");
    calls.clear();
    check(use(&h, MB, b) == GEMM_OK && count("wait") == 1, "the other stream waits for the allocation");
}

// A call that fails behind a launch that works on the buffer.
void failed_call()
{
    gemm_ctx h;
    Stream a, b;
    {
        dg::WorkspaceUse u(&h, handle_of(a));
        check(u.acquire(MB) == GEMM_OK, "acquired");
        calls.clear();
    }
    check(count("record") == 1, "the end of what it launched is recorded");
    {
        dg::WorkspaceUse u(&h, handle_of(b));
        check(u.acquire(64 * MB) == GEMM_OK && calls[1] == "wait" && calls[2] == "freeAsync", "and growth waits for it");
        calls.clear();
        check(u.done() == GEMM_OK && count("record") == 1, "a call that succeeds records its end");
    }
    check(count("record") == 1, "once");
    {
        dg::WorkspaceUse u(&h, handle_of(a));
        calls.clear();
    }
    check(calls.empty(), "a call that uses no workspace records nothing");
}

}  // namespace

int main(int argc, char **argv)
{
    const std::string name = argc > 1 ? argv[1] : "";
    if (name == "growth_in_capture")
        growth_in_capture();
    else if (name == "eager_then_growth_in_capture")
        eager_then_growth_in_capture();
    else if (name == "no_memory_in_capture")
        no_memory_in_capture();
    else if (name == "two_streams")
        two_streams();
    else if (name == "allocated_on_another_stream")
        allocated_on_another_stream();
    else if (name == "failed_call")
        failed_call();
    else
        check(false, "unknown scenario");
    return checks_failed == 0 ? 0 : 1;
}
