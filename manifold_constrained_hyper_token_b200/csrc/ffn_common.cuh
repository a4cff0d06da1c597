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

// bf16 pairs: two floats rounded to one register, and back.
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// v = hi + mid + lo exactly (8 bits each; lo may lose what lies below bf16's
// smallest value): the residual after each rounding to bf16 is an fp32 number.
// Four values, packed in order.  A finite value whose rounding would reach
// infinity is cut instead, and an infinity has no residual; both are rare and
// looked for four at a time.
__device__ __forceinline__ void split3x4(const float4 v, uint2& hi, uint2& mid, uint2& lo) {
  constexpr float kLast = 3.38e38f;  // below bf16's largest value, 3.3895e38
  hi = make_uint2(bf2(v.x, v.y), bf2(v.z, v.w));
  if (fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))) > kLast)
    hi = make_uint2(__float_as_uint(v.x) >> 16 | (__float_as_uint(v.y) & 0xffff0000u),
                    __float_as_uint(v.z) >> 16 | (__float_as_uint(v.w) & 0xffff0000u));
  float r[4] = {v.x - bf_lo(hi.x), v.y - bf_hi(hi.x), v.z - bf_lo(hi.y), v.w - bf_hi(hi.y)};
  if (fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))) > kLast) {
    if (isinf(v.x)) r[0] = 0.0f;
    if (isinf(v.y)) r[1] = 0.0f;
    if (isinf(v.z)) r[2] = 0.0f;
    if (isinf(v.w)) r[3] = 0.0f;
  }
  mid = make_uint2(bf2(r[0], r[1]), bf2(r[2], r[3]));
  lo = make_uint2(bf2(r[0] - bf_lo(mid.x), r[1] - bf_hi(mid.x)),
                  bf2(r[2] - bf_lo(mid.y), r[3] - bf_hi(mid.y)));
}

}  // namespace mhc
