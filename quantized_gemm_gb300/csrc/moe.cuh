// What the two forms of the mixture-of-experts layer share.
#pragma once

#include "kernels.h"
#include "tc_internal.h"

namespace qg {

struct MoeMaps {
  OperandPlan gate, up, down;
};

__device__ __forceinline__ float activate(float g, int act) {
  switch (act) {
    case MM_ACT_SILU: return g / (1.f + expf(-g));
    case MM_ACT_GELU: return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
    default: return g < 0.f ? 0.f : g;   // keeps NaN
  }
}

}  // namespace qg
