// Device helpers of the token operators: eight elements of a row at a time, reductions
// over a row, and the 8-bit format.
#pragma once

#include "dense_device.h"
#include "tokens_internal.h"
#include "wave_route.h"

namespace ecf {

// Eight elements as they lie in memory.
template <class E>
struct Raw8 {
    u32x4_t v[sizeof(typename E::raw) / 2];
};

typedef u32x4_t __attribute__((aligned(2))) u32x4_any2;
typedef u32x4_t __attribute__((aligned(4))) u32x4_any4;

// NT: past the caches, for what is read once
template <class E, bool NT = false>
__device__ __forceinline__ Raw8<E> load_raw8(const typename E::raw *p)
{
    typedef typename std::conditional<sizeof(typename E::raw) == 2, u32x4_any2, u32x4_any4>::type any_t;
    Raw8<E> r;
    if constexpr (NT) {
        r.v[0] = __builtin_nontemporal_load((const any_t *)p);
        if constexpr (sizeof(typename E::raw) == 4)
            r.v[1] = __builtin_nontemporal_load((const any_t *)(p + 4));
    } else if constexpr (sizeof(typename E::raw) == 2) {
        r.v[0] = ((const any128x2 *)p)->v;
    } else {
        r.v[0] = __builtin_bit_cast(u32x4_t, ((const any128x4 *)p)->v);
        r.v[1] = __builtin_bit_cast(u32x4_t, ((const any128x4 *)(p + 4))->v);
    }
    return r;
}

template <class E>
__device__ __forceinline__ void widen8(const Raw8<E> &r, float v[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(typename E::raw) == 2)
            v[j] = E::to_f((uint16_t)(r.v[0][j >> 1] >> (16 * (j & 1))));
        else
            v[j] = __uint_as_float(r.v[j >> 2][j & 3]);
    }
}

// r moved down by s elements (0..8), zeros from above
template <class E>
__device__ __forceinline__ Raw8<E> shift_raw8(Raw8<E> r, int s)
{
    if constexpr (sizeof(typename E::raw) == 2) {
        r.v[0] = s >= 8 ? u32x4_t{0, 0, 0, 0} : shift_down16(r.v[0], s);
    } else {
#pragma unroll
        for (int b = 8; b >= 1; b >>= 1)
            if (s & b) {
                u32x4_t lo = r.v[0], hi = r.v[1];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t x = j + b < 8 ? (j + b < 4 ? lo[(j + b) & 3] : hi[(j + b) & 3]) : 0u;
                    if (j < 4)
                        r.v[0][j] = x;
                    else
                        r.v[1][j - 4] = x;
                }
            }
    }
    return r;
}

// Elements col .. col + 7 (col a multiple of 8) of a row of d, zeros past its end, at any
// alignment of the row.  No lane's load sits behind a branch (d < 8 is the same for all): where the row ends inside
// or before the eight, its last eight are read and moved down.  FULL: d is a multiple of 8,
// and nothing has to be moved.
template <class E, bool FULL, bool NT = false>
__device__ __forceinline__ Raw8<E> row8(const typename E::raw *row, int64_t col, int d)
{
    if constexpr (FULL) {
        Raw8<E> r = load_raw8<E, NT>(row + min(col, (int64_t)d - 8));
        if (col >= d)
#pragma unroll
            for (unsigned i = 0; i < sizeof(r.v) / sizeof(r.v[0]); ++i)
                r.v[i] = u32x4_t{0, 0, 0, 0};
        return r;
    } else {
        if (d >= 8) {
            const int64_t at = min(col, (int64_t)d - 8);
            return shift_raw8<E>(load_raw8<E, NT>(row + at), (int)min(col - at, (int64_t)8));
        }
        Raw8<E> r;
#pragma unroll
        for (unsigned i = 0; i < sizeof(r.v) / sizeof(r.v[0]); ++i)
            r.v[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col == 0 && j < d) {
                if constexpr (sizeof(typename E::raw) == 2)
                    r.v[0][j >> 1] |= (uint32_t)row[j] << (16 * (j & 1));
                else
                    r.v[j >> 2][j & 3] = __float_as_uint(row[j]);
            }
        return r;
    }
}

// This block's number in a block_grid
__device__ __forceinline__ int64_t block_at() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// Sum over the G threads (64, 256 or 1024) that share a row; with G over 64 they are the
// whole block, `sh` has room for one value a wave, and every thread comes here.
template <int G>
__device__ __forceinline__ double row_sum(double v, double *sh)
{
    v = wave_sum_f64(v);
    if constexpr (G > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
            sh[w] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int i = 0; i < G / 64; ++i)
            v += sh[i];
        __syncthreads();
    }
    return v;
}

// ---- 8 bits: e4m3 values over an E8M0 scale per 32 columns -----------------------------

// The scale's byte for a group whose largest finite magnitude has the bits `top`: with
// top = m 2^E, m in [1, 2), and 448 = 1.75 * 2^8, the exponent is E - 8 where m <= 1.75,
// else E - 7; the least scale is 2^-127.
__device__ __forceinline__ int mx_scale_byte(uint32_t top)
{
    return max(0, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
}
// 2^(127 - byte): what the group's values are multiplied by (2^127 .. 2^-120)
__device__ __forceinline__ float mx_inverse(int byte)
{
    return __builtin_ldexpf(1.f, 127 - byte);
}
__device__ __forceinline__ float mx_scale(uint32_t byte)
{
    return byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.f, (int)byte - 127);
}
// Four values as e4m3, to nearest even; finite ones are within 448, or over it by less than its rounding; infinite and
// NaN ones become NaN.
__device__ __forceinline__ uint32_t mx_pack4(const float v[4])
{
    int r = 0;
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (!(fabsf(v[j]) < 449.f))
            r = (r & ~(0xff << (8 * j))) | 0x7f << (8 * j);
    return (uint32_t)r;
}

// ---- launches ------------------------------------------------------------------------

inline dim3 dim_of(BlockGrid g) { return dim3(g.x, g.y); }

// A call of f with types and constants for values
template <class F>
void with_element(int dtype, F f)
{
    if (dtype == ECF_F32)
        f(F32{});
    else if (dtype == ECF_BF16)
        f(BF16{});
    else
        f(F16{});
}
// dtype and another, which is it or ECF_F32
template <class F>
void with_pair(int dtype, int other, F f)
{
    with_element(dtype, [&](auto e) {
        if (other == ECF_F32)
            f(e, F32{});
        else
            f(e, e);
    });
}
template <class F>
void with_bool(bool b, F f)
{
    if (b)
        f(std::true_type{});
    else
        f(std::false_type{});
}

}  // namespace ecf
