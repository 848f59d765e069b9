// The gate of the SwiGLU FFN and its derivative, in fp32.
#pragma once

#include "../device_common.h"

namespace moe {

// act = silu(g) u and, from da = d(loss)/d(act), the gradients of g and u:
//   s = sigmoid(g);  act = g s u;  dg = da u s (1 + g (1 - s));  du = da g s.
// s comes from exp(-g) with the hardware reciprocal (1 ulp).  For very
// negative g, exp(-g) = inf gives s = 0 and act, dg, du their limit 0 (g s
// is -0); for very positive g, 1 - s rounds to 0 and dg = da u.
struct GatedGrad {
    float act, dg, du;
};
__device__ __forceinline__ GatedGrad gated_grad(float g, float u, float da) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    const float gs = g * s;
    return {gs * u, da * u * (s + gs * (1.0f - s)), da * gs};
}

}  // namespace moe
