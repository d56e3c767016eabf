// What the layer operators (moe_host.cpp) need to know of an expert plan whose
// last call was a fused dispatch. Implemented in ep_plan.cpp. Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_kernels.h"
#include "ep.h"

namespace ep {

struct FusedView {
    int32_t M, k, Er, E, H, cap;
    int32_t dtype;            // cfg.combine_dtype
    int32_t wire;             // cfg.combine_wire
    const int32_t* fslot;     // [W][M][k] packed row of a kept first-occurrence slot, else -1
    TokenMap tokens;          // of the last fused dispatch
    bool large;               // a large call (ep_launch_t, combine_row_split)
    bool stream;              // its automatic or given expert cache policy streams
};

// EP_OK and *v, or an error (EP_ERR_NULL, EP_ERR_STATE: no fused dispatch).
int fused_view(const ep_expert_plan_t* plan, const char* call, FusedView* v);
// A kernel reading the plan's map was launched on stream: destroying the plan
// waits for it.
void fused_launched(ep_expert_plan_t* plan, hipStream_t stream);

}  // namespace ep
