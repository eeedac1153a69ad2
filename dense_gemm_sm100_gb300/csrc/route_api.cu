// The C ABI of include/gemm_route.h: argument checks and dispatch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "../../include/gemm.h"
#include "../../include/gemm_route.h"
#include "handle.h"
#include "route.h"

using dg::cuda_fail;
using dg::fail;
using dg::kMaxLd;

namespace {

constexpr int64_t kMaxChoices = int64_t{1} << 30;

int refuse(std::string *why, int code, const char *msg)
{
    if (why) *why = msg;
    return code;
}

int check_logits(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype, int flags,
                 std::string *why)
{
    const auto bad = [&](int code, const char *msg) { return refuse(why, code, msg); };
    if (dtype != GEMM_F32 && dtype != GEMM_BF16) return bad(GEMM_ERR_INVALID, "dtype must be GEMM_F32 or GEMM_BF16");
    if (flags & ~(GEMM_ROUTE_SIGMOID | GEMM_ROUTE_RENORMALISE)) return bad(GEMM_ERR_INVALID, "unknown flags");
    if (experts < 1 || experts > GEMM_ROUTE_MAX_EXPERTS) return bad(GEMM_ERR_INVALID, "experts must be in 1..1024");
    if (k < 1 || k > GEMM_ROUTE_MAX_K || k > experts)
        return bad(GEMM_ERR_INVALID, "k must be in 1..31 and at most the number of experts");
    if (tokens < 0 || tokens > kMaxChoices / k) return bad(GEMM_ERR_INVALID, "tokens * k must be in 0..2^30");
    if (tokens == 0) return GEMM_OK;
    if (!logits) return bad(GEMM_ERR_INVALID, "logits is NULL");
    if (ld < experts || ld > kMaxLd || ld > (int64_t{1} << 44) / tokens)
        return bad(GEMM_ERR_INVALID, "ld must be at least experts and at most 2^36, tokens * ld at most 2^44");
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == GEMM_BF16 ? 2 : 4))
        return bad(GEMM_ERR_ALIGNMENT, "logits is not aligned to its element size");
    return GEMM_OK;
}

int check_route(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
                const float *bias, int64_t groups, int64_t top_groups, int flags, const float *weights,
                const int64_t *expert, const int64_t *order, const int64_t *offsets, std::string *why)
{
    const auto bad = [&](int code, const char *msg) { return refuse(why, code, msg); };
    const int rc = check_logits(tokens, experts, k, logits, ld, dtype, flags, why);
    if (rc) return rc;
    if (groups < 1 || groups > GEMM_ROUTE_MAX_GROUPS || experts % groups)
        return bad(GEMM_ERR_INVALID, "groups must be in 1..32 and divide experts");
    if (top_groups < 1 || top_groups > groups) return bad(GEMM_ERR_INVALID, "top_groups must be in 1..groups");
    if (k > top_groups * (experts / groups)) return bad(GEMM_ERR_INVALID, "k exceeds the experts of top_groups groups");
    if (!offsets) return bad(GEMM_ERR_INVALID, "offsets is NULL");
    if (reinterpret_cast<uintptr_t>(offsets) % 8) return bad(GEMM_ERR_ALIGNMENT, "offsets is not 8-byte aligned");
    if (tokens == 0) return GEMM_OK;
    if (!weights || !expert || !order) return bad(GEMM_ERR_INVALID, "weights, expert or order is NULL");
    if (reinterpret_cast<uintptr_t>(weights) % 4 || reinterpret_cast<uintptr_t>(bias) % 4 ||
        reinterpret_cast<uintptr_t>(expert) % 8 || reinterpret_cast<uintptr_t>(order) % 8)
        return bad(GEMM_ERR_ALIGNMENT, "bias, weights, expert or order is not aligned to its element size");
    return GEMM_OK;
}

int check_grad(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
               const int64_t *expert, const float *dweights, int flags, const void *dlogits, int64_t ldd,
               std::string *why)
{
    const auto bad = [&](int code, const char *msg) { return refuse(why, code, msg); };
    const int rc = check_logits(tokens, experts, k, logits, ld, dtype, flags, why);
    if (rc || tokens == 0) return rc;
    if (!expert || !dweights || !dlogits) return bad(GEMM_ERR_INVALID, "expert, dweights or dlogits is NULL");
    if (ldd < experts || ldd > kMaxLd || ldd > (int64_t{1} << 44) / tokens)
        return bad(GEMM_ERR_INVALID, "ldd must be at least experts and at most 2^36, tokens * ldd at most 2^44");
    if (reinterpret_cast<uintptr_t>(expert) % 8 || reinterpret_cast<uintptr_t>(dweights) % 4 ||
        reinterpret_cast<uintptr_t>(dlogits) % (dtype == GEMM_BF16 ? 2 : 4))
        return bad(GEMM_ERR_ALIGNMENT, "expert, dweights or dlogits is not aligned to its element size");
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_route_validate(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
                        const float *bias, int64_t groups, int64_t top_groups, int flags, float, const float *weights,
                        const int64_t *expert, const int64_t *order, const int64_t *offsets)
{
    return check_route(tokens, experts, k, logits, ld, dtype, bias, groups, top_groups, flags, weights, expert, order,
                       offsets, nullptr);
}

int gemm_route_grad_validate(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
                             const int64_t *expert, const float *dweights, int flags, float, const void *dlogits,
                             int64_t ldd)
{
    return check_grad(tokens, experts, k, logits, ld, dtype, expert, dweights, flags, dlogits, ldd, nullptr);
}

int gemm_route(gemm_handle_t h, int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
               const float *bias, int64_t groups, int64_t top_groups, int flags, float scale, float *weights,
               int64_t *expert, int64_t *order, int64_t *offsets, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    int rc = check_route(tokens, experts, k, logits, ld, dtype, bias, groups, top_groups, flags, weights, expert,
                         order, offsets, &why);
    if (rc) return fail(h, rc, why);
    dg::DeviceGuard guard(h);
    const int sms = h->max_ctas > 0 ? std::min(h->max_ctas, h->sm_count) : h->sm_count;
    dg::RouteArgs a;
    a.logits = logits;
    a.ld = ld;
    a.bf16 = dtype == GEMM_BF16;
    a.tokens = static_cast<int>(tokens);
    a.experts = static_cast<int>(experts);
    a.k = static_cast<int>(k);
    a.bias = bias;
    a.groups = static_cast<int>(groups);
    a.top_groups = static_cast<int>(top_groups);
    a.sigmoid = (flags & GEMM_ROUTE_SIGMOID) != 0;
    a.renormalise = (flags & GEMM_ROUTE_RENORMALISE) != 0;
    a.scale = scale;
    a.weights = weights;
    a.expert = reinterpret_cast<long long *>(expert);
    a.order = reinterpret_cast<long long *>(order);
    a.offsets = reinterpret_cast<long long *>(offsets);
    a.stream = stream;
    dg::WorkspaceUse ws(h, stream);
    const size_t need = tokens > 0 ? dg::route_workspace(tokens, experts, sms) : 0;
    if (need > 0) {
        if ((rc = ws.acquire(need))) return rc;
        a.counts = static_cast<int *>(h->ws);
    }
    int launches = 0;
    const cudaError_t e = dg::launch_route(a, sms, &launches);
    h->launches += launches;
    if (e != cudaSuccess) return cuda_fail(h, e, "router launch");
    h->last_path = tokens == 0 ? "route_empty" : launches == 1 ? "route_one_cta" : "route";
    return ws.done();
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

int gemm_route_grad(gemm_handle_t h, int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld,
                    int dtype, const int64_t *expert, const float *dweights, int flags, float scale, void *dlogits,
                    int64_t ldd, cudaStream_t stream)
try {
    if (!h) return GEMM_ERR_INVALID;
    std::string why;
    const int rc = check_grad(tokens, experts, k, logits, ld, dtype, expert, dweights, flags, dlogits, ldd, &why);
    if (rc) return fail(h, rc, why);
    if (tokens == 0) {
        h->last_path = "noop";
        return GEMM_OK;
    }
    dg::DeviceGuard guard(h);
    dg::RouteGradArgs a;
    a.logits = logits;
    a.ld = ld;
    a.bf16 = dtype == GEMM_BF16;
    a.tokens = static_cast<int>(tokens);
    a.experts = static_cast<int>(experts);
    a.k = static_cast<int>(k);
    a.expert = reinterpret_cast<const long long *>(expert);
    a.dweights = dweights;
    a.sigmoid = (flags & GEMM_ROUTE_SIGMOID) != 0;
    a.renormalise = (flags & GEMM_ROUTE_RENORMALISE) != 0;
    a.scale = scale;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.stream = stream;
    const cudaError_t e = dg::launch_route_grad(a, h->sm_count, h->max_ctas);
    if (e != cudaSuccess) return cuda_fail(h, e, "router gradient launch");
    ++h->launches;
    h->last_path = "route_grad";
    return GEMM_OK;
} catch (...) {
    return GEMM_ERR_NOMEM;  // no exception leaves a C entry
}

}  // extern "C"
