// Device helpers of the dense feed-forward operators: element types and
// activations with their derivatives.
#pragma once

#include <type_traits>

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
    // the hardware's conversion (NaN stays NaN), two values per instruction where they are packed
    static __device__ __forceinline__ raw from_f(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const bf16x2_t v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
};
struct F16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float to_f(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ raw from_f(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return (uint32_t)from_f(a) | (uint32_t)from_f(b) << 16;
    }
};

// v moved down by s 16-bit elements (0..7), zeros from above
__device__ __forceinline__ u32x4_t shift_down16(u32x4_t v, int s)
{
    if (s & 4)
        v = u32x4_t{v[2], v[3], 0, 0};
    if (s & 2)
        v = u32x4_t{v[1], v[2], v[3], 0};
    if (s & 1)
        v = u32x4_t{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    return v;
}

// 8 consecutive elements of a row from column `col` on, at any multiple of their
// size (unaligned 16-byte accesses are one instruction here).  n < 8: the row ends
// after n of them; then the row's last 8 are read and moved down, zeros behind
// them (a row of under 8 elements goes one by one).
struct __attribute__((packed, aligned(2))) any128x2 {
    u32x4_t v;
};
struct __attribute__((packed, aligned(4))) any128x4 {
    f32x4_t v;
};
template <class E>
__device__ __forceinline__ void load8(const void *row, int64_t col, int n, float v[8])
{
    const int s = n >= 8 ? 0 : 8 - n;
    const typename E::raw *q = (const typename E::raw *)row + (col - s);
    if (col >= s) {
        if constexpr (sizeof(typename E::raw) == 4) {
            const f32x4_t a = ((const any128x4 *)q)->v, b = ((const any128x4 *)(q + 4))->v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = a[j], v[4 + j] = b[j];
        } else {
            const u32x4_t a = ((const any128x2 *)q)->v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = E::to_f((uint16_t)(a[j] & 0xffffu));
                v[2 * j + 1] = E::to_f((uint16_t)(a[j] >> 16));
            }
        }
        if (s) {
#pragma unroll
            for (int b = 4; b >= 1; b >>= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (s & b)
                        v[j] = j + b < 8 ? v[j + b] : 0.f;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = j < n ? E::to_f(q[j + s]) : 0.f;
}

// stream: past the caches (non-temporal), for outputs too large to be found there again
template <class E>
__device__ __forceinline__ void store8(void *row, int64_t col, int n, const float v[8], bool stream = false)
{
    typedef f32x4_t __attribute__((aligned(4))) f32x4_a4;
    typedef u32x4_t __attribute__((aligned(2))) u32x4_a2;
    typename E::raw *q = (typename E::raw *)row + col;
    if (n >= 8) {
        if constexpr (sizeof(typename E::raw) == 4) {
            const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
            if (stream) {
                __builtin_nontemporal_store(a, (f32x4_a4 *)q);
                __builtin_nontemporal_store(b, (f32x4_a4 *)(q + 4));
            } else {
                *(f32x4_a4 *)q = a;
                *(f32x4_a4 *)(q + 4) = b;
            }
        } else {
            u32x4_t a;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a[j] = E::pack(v[2 * j], v[2 * j + 1]);
            if (stream)
                __builtin_nontemporal_store(a, (u32x4_a2 *)q);
            else
                *(u32x4_a2 *)q = a;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n)
            q[j] = E::from_f(v[j]);
}

// ---- activations --------------------------------------------------------------------
// exp2 and the reciprocal are the hardware's (within one fp32 step each): with
// expf and a divide, the tanh form's epilogue on 8192 x 16384 outputs cost 100 us
// of 1023, several times what the rounding of the output leaves to see.
//
// Limits hold at the infinities (silu and both gelus: 0 at -inf, inf at +inf) and
// NaN stays NaN: beyond 1e4 each has long become 0 or its argument, so the
// argument of the smooth part stops there, where -inf * 0 would make a NaN.

__device__ __forceinline__ float act_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }

// u2 of silu and of gelu's tanh form, both v / (1 + exp(-u2)):
// 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (v + 0.044715 v^3)
__device__ __forceinline__ float act_u2(float v, int act)
{
    return act == ECF_ACT_SILU ? v : v * (1.5957691216057308f + 0.071354816272600244f * (v * v));
}

// Phi(v) and exp(-v^2/2).  erfc(z) = exp(-z^2) t P(t), t = 1 / (1 + 0.4 z), z = |v| / sqrt 2;
// P of degree 10 is a least-maximum relative fit to exp(z^2) erfc(z) / t, within 6.2e-9 over all z >= 0.
// The product form keeps the relative precision of the negative tail.
__device__ __forceinline__ float act_phi(float v, float &gauss)
{
    const float t = __builtin_amdgcn_rcpf(1.f + 0.28284271247461901f * fabsf(v));
    float p = -0.0292149863f;
    p = p * t + 0.140446045f;
    p = p * t - 0.235525789f;
    p = p * t + 0.13755963f;
    p = p * t - 0.0468938596f;
    p = p * t + 0.0839158009f;
    p = p * t + 0.11900847f;
    p = p * t + 0.171739257f;
    p = p * t + 0.207613732f;
    p = p * t + 0.22567586f;
    p = p * t + 0.225675835f;
    gauss = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
    const float h = 0.5f * t * p * gauss;
    return v < 0.f ? h : 1.f - h;
}

__device__ __forceinline__ float act_value(float v, int act)
{
    if (act == ECF_ACT_NONE)
        return v;
    if (act == ECF_ACT_RELU)
        return v < 0.f ? 0.f : v;
    const float c = v < -1e4f ? -1e4f : v;
    if (act == ECF_ACT_GELU) {
        float gauss;
        return c * act_phi(c, gauss);
    }
    return c * __builtin_amdgcn_rcpf(1.f + act_exp(-act_u2(c, act)));
}

// Value and derivative.  p = 1 / (1 + exp(-u2)); the derivative is
// p + v p (1 - p) u2'(v), with p and 1 - p both from exp(-|u2|) so that neither
// loses its small values.
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
        float gauss;
        const float phi = act_phi(c, gauss);
        value = big * phi;
        slope = phi + c * gauss * 0.39894228040143268f;
        return;
    }
    const float u2 = act_u2(c, act);
    const float du = act == ECF_ACT_SILU ? 1.f : 1.5957691216057308f + 0.21406444881780073f * (c * c);
    const float e = act_exp(-fabsf(u2)), r = __builtin_amdgcn_rcpf(1.f + e);
    const float p = u2 < 0.f ? e * r : r, q = u2 < 0.f ? r : e * r;  // p and 1 - p
    value = big * p;
    slope = p + c * p * q * du;
}

// One branch on the activation for eight values (it is uniform over the launch).
template <class F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case ECF_ACT_NONE: f(std::integral_constant<int, ECF_ACT_NONE>{}); break;
    case ECF_ACT_SILU: f(std::integral_constant<int, ECF_ACT_SILU>{}); break;
    case ECF_ACT_GELU: f(std::integral_constant<int, ECF_ACT_GELU>{}); break;
    case ECF_ACT_GELU_TANH: f(std::integral_constant<int, ECF_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, ECF_ACT_RELU>{}); break;
    }
}

template <class E>
__device__ __forceinline__ const void *row_at(const void *p, int64_t at)
{
    return (const typename E::raw *)p + at;
}
template <class E>
__device__ __forceinline__ void *row_at(void *p, int64_t at)
{
    return (typename E::raw *)p + at;
}

__device__ __forceinline__ void store_el(void *p, int64_t i, float v, int dtype)
{
    if (dtype == ECF_F32)
        ((float *)p)[i] = v;
    else
        ((uint16_t *)p)[i] = dtype == ECF_BF16 ? BF16::from_f(v) : F16::from_f(v);
}

}  // namespace ecf
