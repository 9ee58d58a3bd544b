// Shared by the translation units of the layer behind the router.
#pragma once

#include "internal.h"
#include "moe_router.h"

namespace mr {

// act(g) in fp32: SiLU g / (1 + exp(-g)), or GELU g * Phi(g).
__device__ __forceinline__ float act_f32(float g, int act)
{
    return act == MR_SILU ? g / (1.0f + expf(-g)) : 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
}

// The validation of the forward calls' options (api.cu).
int router_check(const mr_router_params* p);

}  // namespace mr
