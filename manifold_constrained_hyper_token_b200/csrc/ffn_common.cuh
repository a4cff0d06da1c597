// ffn_common.cuh -- what the feed-forward block's kernels share: the gate
// activation and its derivative, and the exact split of an fp32 value into
// three bf16 parts.
#pragma once

#include "mhc_common.cuh"

namespace mhc {

// act(g) and act'(g).  FAST (bf16 results, rounded to 8 bits right after): the
// exponential and the quotient by their approximate instructions, each good to
// about 2^-21, against a rounding of 2^-9; otherwise the accurate functions.
template <bool FAST>
__device__ __forceinline__ void gate_both(int act, float g, float& h, float& dh) {
  if (act == MHC_ACT_SILU) {
    const float p = FAST ? __fdividef(1.0f, 1.0f + __expf(-g)) : 1.0f / (1.0f + expf(-g));
    h = g * p;
    dh = fmaf(h, 1.0f - p, p);
  } else {
    const float c = 0.5f * erfcf(-0.70710678118654752f * g);
    const float e = FAST ? __expf(-0.5f * g * g) : expf(-0.5f * g * g);
    h = g * c;
    dh = fmaf(g * 0.39894228040143268f, e, c);
  }
}
template <bool FAST> __device__ __forceinline__ float gate(int act, float g) {
  if (act == MHC_ACT_SILU)
    return FAST ? __fdividef(g, 1.0f + __expf(-g)) : g / (1.0f + expf(-g));
  return g * (0.5f * erfcf(-0.70710678118654752f * g));
}

// v = hi + mid + lo exactly (8 bits each; lo may lose what lies below bf16's
// smallest value): the residual after each rounding to bf16 is an fp32 number.
// A finite v whose rounding would reach infinity is cut instead; a non-finite v
// has no residual.
__device__ __forceinline__ void split3(float v, float& hi, float& mid, float& lo) {
  hi = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(hi) && !isinf(v)) hi = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  const float r = isfinite(hi) ? v - hi : 0.0f;
  mid = __bfloat162float(__float2bfloat16_rn(r));
  lo = r - mid;
}

}  // namespace mhc
