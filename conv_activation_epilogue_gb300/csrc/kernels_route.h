// kernels_route.h -- host-side view of the router's kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mmact {

constexpr int ROUTE_MAX_TOP = 16, ROUTE_MAX_EXPERTS = 512;

struct RouteArgs {
    int64_t T;
    int E, top, normalize;
    float coef;
    const void *logits;          // [T, E]
    const uint8_t *mask;         // [T] or null
    int *experts;                // [T, top]
    float *probs;                // [T, top]
    int *counts;                 // [E + 1]
    float *loss;                 // [1]
    // workspace: of each CTA, sums of softmax over its tokens [grid, E], slots [grid, E + 1]
    float *part;
    int *part_counts;
};

struct RouteBackwardArgs {
    int64_t T;
    int E, top, normalize;
    float coef;
    const void *logits;
    const uint8_t *mask;
    const int *experts, *counts;
    const float *dprobs;         // [T, top] or null
    const float *dloss;          // [1] or null
    void *dlogits;               // [T, E]
};

int route_grid(int64_t T, int64_t E, int64_t top, int sms);        // CTAs of the forward pass
cudaError_t launch_moe_route(const RouteArgs &a, int type, int grid, int sms, cudaStream_t s);   // grid of route_grid
cudaError_t launch_moe_route_backward(const RouteBackwardArgs &a, int type, int sms, cudaStream_t s);

}  // namespace mmact
