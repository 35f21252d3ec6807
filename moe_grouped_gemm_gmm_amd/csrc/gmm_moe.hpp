// Internal launchers of the router, the order of the slots by expert and the
// rows moved there and back (include/gmm_moe.h).  Arguments are already
// validated by gmm_moe_api.cpp; each launcher only enqueues kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

struct RouteArgs {
    const void* logits;       // [T,E]
    const float* bias;        // [E] or NULL
    int64_t T;
    int E, k;
    bool sigmoid, normalize;
    float scale;
};
hipError_t launch_route(const RouteArgs& a, bool logits_bf16, int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_route_bwd(const RouteArgs& a, bool logits_bf16, const float* dweights, const int32_t* ids,
                            void* dlogits, bool out_bf16, hipStream_t stream);

// The order of n slots by expert; `counts` holds sort_count_words(n, G) int32.
int64_t sort_count_words(int64_t n, int64_t G);
hipError_t launch_sort_tokens(const int32_t* ids, int n, int first, int G, int M, int32_t* group_sizes,
                              int32_t* row_of, int32_t* slot_of, int32_t* counts, int32_t* status, hipStream_t stream);

struct MoveArgs {
    const int32_t *row_of, *slot_of;   // [T,k], [M]
    const float* weights;              // [T,k] or NULL
    int64_t T, M;
    int k;
    int64_t K;                         // a multiple of 8
};
hipError_t launch_dispatch(const MoveArgs& a, const void* x, bool bf16, void* out, hipStream_t stream);
hipError_t launch_combine(const MoveArgs& a, const void* y, bool y_bf16, const void* residual, void* out,
                          bool out_bf16, hipStream_t stream);
hipError_t launch_combine_bwd(const MoveArgs& a, const void* dout, bool dout_bf16, const void* y, bool y_bf16,
                              void* dy, float* dweights, hipStream_t stream);

}  // namespace gmm
