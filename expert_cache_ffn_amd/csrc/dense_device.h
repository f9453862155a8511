// Device helpers of the dense feed-forward operators: element types and
// activations with their derivatives.
#pragma once

#include "dense_internal.h"
#include "device_common.h"

namespace ecf {

// Element types: fp32, bf16 and fp16 (IEEE half).  to_f widens exactly, from_f
// rounds to nearest even.
struct F32 {
    typedef float raw;
    static __device__ __forceinline__ float to_f(raw v) { return v; }
    static __device__ __forceinline__ raw from_f(float v) { return v; }
};
struct BF16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float to_f(raw v) { return bf_to_f(v); }
    static __device__ __forceinline__ raw from_f(float v) { return f_to_bf(v); }
};
struct F16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float to_f(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ raw from_f(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};

// Value of the activation.  The limits hold at the infinities (silu and both
// gelus: 0 at -inf, inf at +inf) and NaN stays NaN: below -1e4 every one of
// them has underflowed to zero, so the argument stops there, where -inf * 0
// would make a NaN.
//   gelu       0.5 v erfc(-v / sqrt 2): erfc keeps the relative precision of the negative tail
//   gelu_tanh  0.5 v (1 + tanh u) = v / (1 + exp(-2 u)), u = sqrt(2/pi) (v + 0.044715 v^3)
__device__ __forceinline__ float act_value(float v, int act)
{
    if (act == ECF_ACT_NONE)
        return v;
    if (act == ECF_ACT_RELU)
        return v < 0.f ? 0.f : v;
    const float c = v < -1e4f ? -1e4f : v;
    if (act == ECF_ACT_GELU)
        return 0.5f * c * erfcf(c * -0.70710678118654752f);
    const float u2 = act == ECF_ACT_SILU ? c : c * (1.5957691216057308f + 0.071354816272600244f * (c * c));
    return c / (1.f + expf(-u2));
}

// Value and derivative.  p = 1 / (1 + exp(-u2)); the derivative is
// p + v p (1 - p) u2'(v), whose second term is dropped where p (1 - p)
// underflows, so that infinities give the limits 0 and 1.
__device__ __forceinline__ void act_both(float v, int act, float &value, float &slope)
{
    if (act == ECF_ACT_NONE) {
        value = v;
        slope = 1.f;
        return;
    }
    if (act == ECF_ACT_RELU) {
        value = v < 0.f ? 0.f : v;
        slope = v > 0.f ? 1.f : v != v ? v : 0.f;
        return;
    }
    const float c = v < -1e4f ? -1e4f : v > 1e4f ? 1e4f : v;
    const float big = v > 1e4f ? v : c;  // the value keeps growing with v
    if (act == ECF_ACT_GELU) {
        const float cdf = 0.5f * erfcf(c * -0.70710678118654752f);
        value = big * cdf;
        slope = cdf + c * expf(-0.5f * c * c) * 0.39894228040143268f;
        return;
    }
    const float u2 = act == ECF_ACT_SILU ? c : c * (1.5957691216057308f + 0.071354816272600244f * (c * c));
    const float du = act == ECF_ACT_SILU ? 1.f : 1.5957691216057308f + 0.21406444881780073f * (c * c);
    const float e = expf(-fabsf(u2)), r = 1.f / (1.f + e);
    const float p = u2 < 0.f ? e * r : r, q = u2 < 0.f ? r : e * r;  // p and 1 - p
    value = big * p;
    slope = p + c * p * q * du;
}

}  // namespace ecf
