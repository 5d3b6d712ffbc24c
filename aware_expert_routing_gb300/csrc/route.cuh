// route.cuh -- the selection of moe_select_params: its arguments and launchers
// (route.cu).  Apart from common.cuh, which is part of what identifies the
// expert kernel's code in its profile records.
#pragma once

#include "common.cuh"

namespace moe {

// Selection of moe_select_params (top-k mode only).
struct SelectArgs {
    const float* bias;      // [N] or null, added to the selection values
    int sigmoid;            // 1: sigmoid scores, 0: softmax
    int n_group, topk_group, group_top;
    int renorm;
    float scale;
};

cudaError_t launch_route(const RouteArgs& a, const SelectArgs& sel, cudaStream_t s);
cudaError_t launch_route_fused(const RouterArgs& r, const RouteArgs& a, const SelectArgs& sel, cudaStream_t s);

}  // namespace moe
