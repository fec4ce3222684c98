// What the two forms of the mixture-of-experts layer share.
#pragma once

#include "kernels.h"
#include "tc_internal.h"

namespace qg {

struct MoeMaps {
  OperandPlan gate, up, down;
};

// 1 + erf(z) = erfc(-z), which keeps its digits where erf is close to -1.  Not
// inlined: the epilogues unroll it 16 times, and its code then slows a short
// layer's start (3 tokens, 12 picks of K = 1000, F = 712: GELU 32.5 us inlined;
// SiLU 31.8 inlined).
static __device__ __noinline__ float gelu(float g) { return 0.5f * g * erfcf(g * -0.70710678118654752f); }

__device__ __forceinline__ float activate(float g, int act) {
  switch (act) {
    case MM_ACT_SILU: return g / (1.f + expf(-g));
    case MM_ACT_GELU: return gelu(g);
    default: return g < 0.f ? 0.f : g;   // keeps NaN
  }
}

}  // namespace qg
