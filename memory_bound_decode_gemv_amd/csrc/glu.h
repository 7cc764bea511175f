// glu.h -- the epilogue of the gated feed-forward products: y = act(g) * u from
// the binary32 sums of a gate row and an up row.  Device code only.
//
// SiLU and the tanh form of GELU are written as g / (1 + exp(-z)) (tanh(z/2) =
// 2 / (1 + exp(-z)) - 1), and GELU with erfc, so that no branch subtracts
// nearly equal numbers: for very negative g each tends to zero with the
// relative accuracy of exp and erfc (exp(-z) = infinity gives the signed zero).
#pragma once

#include "decodegemv.h"
#include "dg_device.h"

namespace dg {

// What a kernel's GLU form takes besides the plain form's arguments; the plain
// form takes nothing.
template <bool GLU>
struct GluArgs {};
template <>
struct GluArgs<true> {
    const uint8_t* Wu;   // the up matrix, laid out like the gate's
    int act;             // DG_ACT_*
};

__device__ __forceinline__ float glu_act(int act, float g) {
    if (act == DG_ACT_RELU) return g < 0.0f ? 0.0f : g;
    if (act == DG_ACT_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
    const float z = act == DG_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-z));
}

__device__ __forceinline__ float glu(int act, float g, float u) { return glu_act(act, g) * u; }

}  // namespace dg
