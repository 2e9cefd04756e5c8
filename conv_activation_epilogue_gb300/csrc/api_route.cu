// api_route.cu -- the C ABI of the router in training (include/mmact.h): argument
// validation and launches.  As in api.cu, every check happens on the host before
// anything is enqueued.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "api_checks.h"
#include "api_internal.h"
#include "kernels_route.h"
#include "mmact.h"

#define MMACT_EXPORT extern "C" __attribute__((visibility("default")))

namespace mmact {
namespace {

mmact_status route_sizes(int64_t T, int64_t E, int64_t top)
{
    if (T < 0 || E < 0 || top < 0 || T > MAX_DIM) return MMACT_ERR_INVALID_ARG;
    if (E < 1 || E > ROUTE_MAX_EXPERTS || top < 1 || top > ROUTE_MAX_TOP || top > E) return MMACT_ERR_UNSUPPORTED;
    if (T * top > MAX_DIM) return MMACT_ERR_UNSUPPORTED;       // an expert's slots are counted in 32 bits
    return MMACT_OK;
}

// Partial results of as many CTAs as there can be: 8 tokens to a CTA at least (8 warps, a
// whole one to a token at most), one for each SM of a device of 512 at most.  A
// workspace's size depends on T and E alone.
constexpr int ROUTE_MAX_SMS = 512;
int64_t route_max_grid(int64_t T) { return std::min<int64_t>((T + 7) / 8, ROUTE_MAX_SMS); }
int64_t route_part_bytes(int64_t grid, int64_t E) { return round_up(grid * E * 4, 256); }

}  // namespace
}  // namespace mmact

using namespace mmact;

MMACT_EXPORT mmact_status mmact_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t *bytes)
{
    if (bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    const mmact_status s = route_sizes(T, E, 1);
    if (s != MMACT_OK) return s;
    const int64_t grid = route_max_grid(T);
    *bytes = route_part_bytes(grid, E) + grid * (E + 1) * 4;
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_moe_route(const void *logits, const uint8_t *mask, int32_t *experts, float *probs,
                                          int32_t *counts, float *loss, int64_t T, int64_t E, int64_t top,
                                          mmact_dtype logits_dtype, int normalize, float coef, void *workspace, void *stream)
{
    if (!valid_float(logits_dtype)) return MMACT_ERR_INVALID_ARG;
    mmact_status s = route_sizes(T, E, top);
    if (s != MMACT_OK) return s;
    if (counts == nullptr || loss == nullptr) return MMACT_ERR_INVALID_ARG;
    if (T != 0 && (logits == nullptr || experts == nullptr || probs == nullptr || workspace == nullptr))
        return MMACT_ERR_INVALID_ARG;
    if (!aligned4(experts) || !aligned4(probs) || !aligned4(counts) || !aligned4(loss)) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(workspace)) return MMACT_ERR_UNSUPPORTED;
    DeviceContext dev;
    if ((s = device_context(&dev)) != MMACT_OK) return s;
    const int sms = std::min(dev.sm_count, ROUTE_MAX_SMS), grid = route_grid(T, E, top, sms);
    RouteArgs a;
    a.T = T;
    a.E = (int)E;
    a.top = (int)top;
    a.normalize = normalize != 0;
    a.coef = coef;
    a.logits = logits;
    a.mask = mask;
    a.experts = experts;
    a.probs = probs;
    a.counts = counts;
    a.loss = loss;
    a.part = static_cast<float *>(workspace);
    a.part_counts = reinterpret_cast<int *>(static_cast<char *>(workspace) + route_part_bytes(grid, E));
    return enqueued(launch_moe_route(a, out_kind(logits_dtype), grid, sms, static_cast<cudaStream_t>(stream)));
}

MMACT_EXPORT mmact_status mmact_moe_route_backward(const void *logits, const uint8_t *mask, const int32_t *experts,
                                                   const int32_t *counts, const float *dprobs, const float *dloss,
                                                   void *dlogits, int64_t T, int64_t E, int64_t top, mmact_dtype logits_dtype,
                                                   int normalize, float coef, void *stream)
{
    if (!valid_float(logits_dtype)) return MMACT_ERR_INVALID_ARG;
    mmact_status s = route_sizes(T, E, top);
    if (s != MMACT_OK) return s;
    if (T == 0) return MMACT_OK;
    if (logits == nullptr || counts == nullptr || dlogits == nullptr || (dprobs != nullptr && experts == nullptr))
        return MMACT_ERR_INVALID_ARG;
    if (!aligned4(experts) || !aligned4(counts) || !aligned4(dprobs) || !aligned4(dloss)) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(dlogits)) return MMACT_ERR_UNSUPPORTED;
    DeviceContext dev;
    if ((s = device_context(&dev)) != MMACT_OK) return s;
    RouteBackwardArgs a;
    a.T = T;
    a.E = (int)E;
    a.top = (int)top;
    a.normalize = normalize != 0;
    a.coef = coef;
    a.logits = logits;
    a.mask = mask;
    a.experts = experts;
    a.counts = counts;
    a.dprobs = dprobs;
    a.dloss = dloss;
    a.dlogits = dlogits;
    return enqueued(launch_moe_route_backward(a, out_kind(logits_dtype), dev.sm_count, static_cast<cudaStream_t>(stream)));
}
