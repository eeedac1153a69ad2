// Launch interface of the expert router (route.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dg {

struct RouteArgs {
    const void *logits = nullptr;
    long long ld = 0;
    bool bf16 = false;
    int tokens = 0, experts = 0, k = 0;
    const float *bias = nullptr;  // null: none
    int groups = 1, top_groups = 1;
    bool sigmoid = false, renormalise = false;
    float scale = 1.0f;
    float *weights = nullptr;
    long long *expert = nullptr, *order = nullptr, *offsets = nullptr;
    int *counts = nullptr;  // workspace: route_workspace() bytes
    cudaStream_t stream = nullptr;
};

// CTAs that route (each a run of tokens); one: no workspace, one launch.
int route_chunks(int64_t tokens, int sm_count);
size_t route_workspace(int64_t tokens, int64_t experts, int sm_count);
// *launches: kernels launched.
cudaError_t launch_route(const RouteArgs &a, int sm_count, int *launches);

struct RouteGradArgs {
    const void *logits = nullptr;
    long long ld = 0;
    bool bf16 = false;
    int tokens = 0, experts = 0, k = 0;
    const long long *expert = nullptr;
    const float *dweights = nullptr;
    bool sigmoid = false, renormalise = false;
    float scale = 1.0f;
    void *dlogits = nullptr;
    long long ldd = 0;
    cudaStream_t stream = nullptr;
};
cudaError_t launch_route_grad(const RouteGradArgs &a, int sm_count, int max_ctas);

}  // namespace dg
