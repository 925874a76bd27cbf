// What the kernels of the gated feed-forward product share: h = act(g) u, g = x Wg^T, u = x Wu^T.
#pragma once

#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace glu {

// act(g) and its derivative.  SiLU: g s, s + g s (1 - s).  GELU: g Phi(g), Phi(g) + g phi(g), Phi the normal distribution.
struct Act {
    float v, d;
};
__device__ __forceinline__ float act(float g, bool gelu) { return gelu ? g * normcdff(g) : g * sigmoid(g); }
__device__ __forceinline__ Act act_and_slope(float g, bool gelu) {
    if (gelu) {
        const float c = normcdff(g);
        return {g * c, fmaf(g * 0.3989422804014327f, expf(-0.5f * g * g), c)};
    }
    const float s = sigmoid(g), gs = g * s;
    return {gs, s + gs - gs * s};
}

}  // namespace glu
}  // namespace mixer
