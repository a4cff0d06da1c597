// ffn_common.cuh -- what the feed-forward block's kernels share: the gate
// activation and its derivative, and the exact split of an fp32 value into
// three bf16 parts.
#pragma once

#include "mhc_common.cuh"

namespace mhc {

// act(g) and act'(g).  FAST (bf16 results, rounded to 8 bits right after): the
// exponential and the quotient by their approximate instructions.  The quotient is
// good to 2^-22; the exponential's error grows with its argument, 2 + 1.2 |g| units of
// 2^-24: 2^-20 of the sigmoid at |g| = 12 and 2^-17 at 80, against a rounding of 2^-9.
// Otherwise the accurate functions.
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

// Two floats rounded to a bf16 pair.
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// v = hi + mid + lo exactly, three bf16 numbers of 8 bits each (lo may lose what
// lies below bf16's smallest value).  The upper half of an fp32 number is the
// bf16 number it is cut to, so each plane is a mask and a subtraction; cutting
// rather than rounding leaves mid below 2^-7 of v and lo below 2^-15, and cannot
// overflow.  Non-finite values stay non-finite.  Four values, packed in order.
__device__ __forceinline__ void split3x4(const float4 v, uint2& hi, uint2& mid, uint2& lo) {
  const float in[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __float_as_uint(in[i]);
    const float r = in[i] - __uint_as_float(h[i] & 0xffff0000u);
    m[i] = __float_as_uint(r);
    l[i] = __float_as_uint(r - __uint_as_float(m[i] & 0xffff0000u));
  }
  hi = make_uint2(__byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
  mid = make_uint2(__byte_perm(m[0], m[1], 0x7632), __byte_perm(m[2], m[3], 0x7632));
  lo = make_uint2(__byte_perm(l[0], l[1], 0x7632), __byte_perm(l[2], l[3], 0x7632));
}

}  // namespace mhc
