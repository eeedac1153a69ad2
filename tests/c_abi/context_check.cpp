// The context that a call works in (DeviceGuard of csrc/handle.h) against a model
// of the driver's and the runtime's notion of a current context, on the CPU.
// Usage: context_check <scenario>; exit code 0 when every check holds.
#include <cstdio>
#include <cstring>

#include "handle.h"

namespace {

// Contexts of the model: a device, and whether it is that device's primary one.
struct Context {
    int device;
};
Context primary[2] = {{0}, {1}}, own[2] = {{0}, {1}};
Context *current = nullptr;  // the thread's
int runtime_device = 0;      // what the runtime reports where there is none
int sets = 0, checks_failed = 0;

CUcontext handle_of(Context *c) { return reinterpret_cast<CUcontext>(c); }

void check(bool ok, const char *what)
{
    if (ok) return;
    std::printf("failed: %s\n", what);
    ++checks_failed;
}

CUresult CUDAAPI get_context(CUcontext *c)
{
    *c = handle_of(current);
    return CUDA_SUCCESS;
}

CUresult CUDAAPI set_context(CUcontext c)
{
    current = reinterpret_cast<Context *>(c);
    ++sets;
    return CUDA_SUCCESS;
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 dg::g_encode = nullptr;
PFN_cuCtxGetCurrent_v4000 dg::g_get_context = get_context;
PFN_cuCtxSetCurrent_v4000 dg::g_set_context = set_context;

extern "C" {

cudaError_t cudaGetLastError(void) { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "an error of the model"; }

cudaError_t cudaGetDevice(int *d)
{
    *d = current ? current->device : runtime_device;
    return cudaSuccess;
}

cudaError_t cudaSetDevice(int d)
{
    runtime_device = d;
    current = &primary[d];
    ++sets;
    return cudaSuccess;
}

}  // extern "C"

namespace {

gemm_ctx made_in(Context *c)
{
    gemm_ctx h;
    h.device = c->device;
    h.context = handle_of(c);
    return h;
}

// Inside a call the handle's context is current, behind it the thread's.
void call(const gemm_ctx &h, Context *after)
{
    {
        dg::DeviceGuard guard(&h);
        check(handle_of(current) == h.context, "the handle's context is current in a call");
    }
    check(current == after, "the thread's context is back behind it");
}

void same()
{
    for (Context *c : {&primary[0], &own[0]}) {
        current = c;
        sets = 0;
        call(made_in(c), c);
        check(sets == 0, "nothing is set where the handle's context is current");
    }
}

void other()
{
    for (Context *mine : {&own[0], &primary[1], &own[1]}) {
        current = mine;
        call(made_in(&primary[0]), mine);
    }
    current = &primary[0];
    call(made_in(&own[0]), &primary[0]);
}

void none()
{
    current = nullptr;
    call(made_in(&primary[0]), &primary[0]);  // as any CUDA call leaves it
    current = nullptr;
    runtime_device = 0;
    call(made_in(&primary[1]), &primary[0]);
}

void making()
{
    for (Context *mine : {&own[0], &primary[0]}) {
        current = mine;
        dg::DeviceGuard guard(0);
        check(current == mine, "a handle is made in the thread's own context of its device");
    }
    current = &own[0];
    {
        dg::DeviceGuard guard(1);
        check(current == &primary[1], "or in the primary one of another device");
    }
    check(current == &own[0], "which leaves the thread's as it was");
    current = nullptr;
    runtime_device = 0;
    {
        dg::DeviceGuard guard(0);
        check(current == &primary[0], "or in the primary one where the thread has none");
    }
    check(current == &primary[0], "which it keeps");
}

}  // namespace

int main(int argc, char **argv)
{
    const char *what = argc > 1 ? argv[1] : "";
    if (!std::strcmp(what, "same")) same();
    else if (!std::strcmp(what, "other")) other();
    else if (!std::strcmp(what, "none")) none();
    else if (!std::strcmp(what, "making")) making();
    else return 2;
    return checks_failed ? 1 : 0;
}
