// Root-mean-square norm with the residual's addition, forward and backward.
//
// Forward: s = x + residual (rounded to its type), y = s * rstd * w with
// rstd = 1 / sqrt(mean s^2 + eps).  A row is read once: its threads hold it in registers
// over the sum of squares, which is taken in 64 bits (an fp32 square overflows at values of
// 1.8e19 that bf16 and fp32 hold).  8 bits: four lanes have the 32 columns of a scale, so
// its maximum is two DPP steps.
//
// Backward: with h = s rstd and g = dy w, ds = dsum + rstd (g - h mean(g h)), and
// dw = sum_t dy h.  A group of threads walks over rows, holding its columns' part of dw in
// registers; the parts are joined in a fixed order by a second kernel.
//
// A row has as many threads as hold it in at most four chunks of eight elements each: a
// wave of its own up to 1024 elements needs no barrier, four waves up to 8192, sixteen up to
// 16384.  Longer rows are read again from the caches.
//
// Bound by memory.  bf16 with an fp32 sum: 8192 x 4096 to 8 bits 70 us (5.2 TB/s, where a large
// copy takes 5.0), 4096 x 4096 backward 46 us and 5 for the join (5.8 TB/s); one token of
// 4096 3.1 us, launch and two rounds of loads.  Backward over rows of 8193 to 16384 the sixteen
// waves have 128 registers a thread, which 16-bit types spill over (9 or 10 registers with an fp32 sum, 43
// without): 4096 x 16384 219 us with an fp32 sum (4.9 TB/s), fp32 211 (5.1), bf16 throughout 141
// (3.8 TB/s, so not at memory's rate).
#include "tokens_device.h"

namespace ecf {
namespace {

constexpr int kNormWide = 16384;  // longer rows are read again instead of held

struct NormPlan {
    int group, chunks;  // threads per row, chunks of 8 elements each holds (0: a loop)
};
// Rows to threads: a wave up to 1024 elements, four up to 8192, sixteen above.
NormPlan norm_plan(int d)
{
    if (d <= 512)
        return {64, 1};
    if (d <= 1024)
        return {64, 2};
    if (d <= 2048)
        return {256, 1};
    if (d <= 4096)
        return {256, 2};
    if (d <= 8192)
        return {256, 4};
    return {1024, d <= kNormWide ? 2 : 0};
}

// 1 / sqrt(v) by the hardware's estimate and one Newton step in 64 bits
__device__ __forceinline__ float inverse_root(double v)
{
    const double r = __builtin_amdgcn_rsq(v);
    return (float)(v > 0.0 && v < __builtin_inf() ? r * fma(-0.5 * v, r * r, 1.5) : r);
}

template <class W>
__device__ __forceinline__ void weight8(const NormCall &c, int64_t col, float w[8])
{
    if (c.weight) {
        widen8<W>(row8<W, false>((const typename W::raw *)c.weight, col, c.d), w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = 1.f;
    }
}
template <class E>
__device__ __forceinline__ void weight8_of(const NormCall &c, int64_t col, float w[8])
{
    if (c.weight_dtype == ECF_F32)
        weight8<F32>(c, col, w);
    else
        weight8<E>(c, col, w);
}

// Eight elements of y, from s, w and v = mean s^2 + eps, to their outputs.  Every lane comes
// here: four share a scale.
template <class E>
__device__ __forceinline__ void put_y(const NormCall &c, int64_t t, int64_t col, const float s[8], const float w[8], float rstd,
                                      double v)
{
    const int n = (int)max((int64_t)0, min((int64_t)8, c.d - col));
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] = s[j] * rstd * w[j];
    if (c.y)
        store8<E>((typename E::raw *)c.y + t * c.ldy, col, n, y);
    if (!c.q)
        return;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(y[j]) & 0x7fffffffu;
        top = max(top, b < 0x7f800000u ? b : 0u);
    }
    top = max(top, dpp32<kDppXor1>(top));
    top = max(top, dpp32<kDppXor2>(top));
    int byte = mx_scale_byte(top);
    // y has three fp32 roundings, 2.6 steps of its value near a border.  Where they leave open on which side of
    // 1.75 2^E the largest one lies, (s w)^2 is compared with (1.75 2^E)^2 v in 64 bits (by all four lanes).
    if ((top & 0x7fffffu) - 0x5ffffcu <= 8u) {
        const double border = (double)__uint_as_float((top & 0x7f800000u) | 0x600000u), most = border * border * v;
        uint32_t over = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float sj = s[j];
            asm volatile("" : "+v"(sj));  // (or s stays in registers in 64 bits from the sum of squares on: 156 registers for four chunks, not 103)
            const double p = (double)sj * (double)w[j];
            over |= fabsf(y[j]) < __builtin_inff() && p * p > most;
        }
        over |= dpp32<kDppXor1>(over);
        over |= dpp32<kDppXor2>(over);
        byte = mx_scale_byte((top & 0x7f800000u) | (0x600000u + over));
    }
    const float inv = mx_inverse(byte);
    float scaled[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        scaled[j] = y[j] * inv;
    uint32_t p[2] = {mx_pack4(scaled), mx_pack4(scaled + 4)};
    uint8_t *q = (uint8_t *)c.q + t * c.ldq + col;
    if (n == 8) {
        struct __attribute__((packed, aligned(1))) any64 {
            uint32_t v[2];
        };
        *(any64 *)q = any64{{p[0], p[1]}};
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n)
                q[j] = (uint8_t)(p[j >> 2] >> (8 * (j & 3)));
    }
    if ((threadIdx.x & 3) == 0 && n > 0)
        ((uint8_t *)c.q_scale)[t * c.ldqs + col / 32] = (uint8_t)byte;
}

// s of a chunk, rounded to its type
template <class E, class S, bool FULL>
__device__ __forceinline__ void sum8(const Raw8<E> &x, const Raw8<S> &r, bool has, float s[8])
{
    widen8<E>(x, s);
    if (has) {
        float q[8];
        widen8<S>(r, q);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = S::to_f(S::from_f(s[j] + q[j]));
    }
}

// grid: one group of G threads per row
template <class E, class S, int G, int NC, bool FULL>
__global__ __launch_bounds__(G > 256 ? G : 256) void k_norm(NormCall c)
{
    __shared__ double sh[16];
    constexpr int B = G > 256 ? G : 256;
    const int64_t t = block_at() * (B / G) + threadIdx.x / G;
    if (t >= c.T)
        return;  // (whole waves, where a wave has a row of its own, or whole blocks)
    const int i = threadIdx.x % G;
    const typename E::raw *x = (const typename E::raw *)c.x + t * c.ldx;
    const typename S::raw *res = (const typename S::raw *)c.residual + t * c.ldres;
    Raw8<E> xr[NC];
    Raw8<S> rr[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k)
        xr[k] = row8<E, FULL>(x, (int64_t)(k * G + i) * 8, c.d);
    if (c.residual)
#pragma unroll
        for (int k = 0; k < NC; ++k)
            rr[k] = row8<S, FULL>(res, (int64_t)(k * G + i) * 8, c.d);
    float w[NC][8], s[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k)
        weight8_of<E>(c, (int64_t)(k * G + i) * 8, w[k]);
    double q = 0.0;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        sum8<E, S, FULL>(xr[k], rr[k], c.residual, s[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q = fma((double)s[k][j], (double)s[k][j], q);
    }
    q = row_sum<G>(q, sh);
    const double v = q / c.d + (double)c.eps;
    const float rstd = inverse_root(v);
    if (i == 0 && c.rstd)
        c.rstd[t] = rstd;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int64_t col = (int64_t)(k * G + i) * 8;
        if (c.sum)
            store8<S>((typename S::raw *)c.sum + t * c.ldsum, col, (int)max((int64_t)0, min((int64_t)8, c.d - col)), s[k]);
        put_y<E>(c, t, col, s[k], w[k], rstd, v);
    }
}

// Rows of any length, one block each: the sum is written in the first pass and read back
// by the thread that wrote it (or taken anew from x).  Where the sum is the residual, a load
// of the row's last eight may see elements that other threads have written: row8 drops them.
template <class E, class S>
__global__ __launch_bounds__(1024) void k_norm_wide(NormCall c)
{
    __shared__ double sh[16];
    const int64_t t = block_at();
    if (t >= c.T)
        return;
    const typename E::raw *x = (const typename E::raw *)c.x + t * c.ldx;
    const typename S::raw *res = (const typename S::raw *)c.residual + t * c.ldres;
    typename S::raw *sum = (typename S::raw *)c.sum + t * c.ldsum;
    const int rounds = (c.d + 8 * 1024 - 1) / (8 * 1024);
    double q = 0.0;
    for (int k = 0; k < rounds; ++k) {
        const int64_t col = ((int64_t)k * 1024 + threadIdx.x) * 8;
        Raw8<S> r{};
        if (c.residual)
            r = row8<S, false>(res, col, c.d);
        float s[8];
        sum8<E, S, false>(row8<E, false>(x, col, c.d), r, c.residual, s);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q = fma((double)s[j], (double)s[j], q);
        if (c.sum)
            store8<S>(sum, col, (int)max((int64_t)0, min((int64_t)8, c.d - col)), s);
    }
    q = row_sum<1024>(q, sh);
    const double v = q / c.d + (double)c.eps;
    const float rstd = inverse_root(v);
    if (threadIdx.x == 0 && c.rstd)
        c.rstd[t] = rstd;
    for (int k = 0; k < rounds; ++k) {
        const int64_t col = ((int64_t)k * 1024 + threadIdx.x) * 8;
        float s[8], w[8];
        if (c.sum) {
            widen8<S>(row8<S, false>(sum, col, c.d), s);
        } else {
            Raw8<S> r{};
            if (c.residual)
                r = row8<S, false>(res, col, c.d);
            sum8<E, S, false>(row8<E, false>(x, col, c.d), r, c.residual, s);
        }
        weight8_of<E>(c, col, w);
        put_y<E>(c, t, col, s, w, rstd, v);
    }
}

template <class E, class S>
__device__ __forceinline__ void put_ds(const NormCall &c, int64_t t, int64_t col, const float v[8])
{
    const int n = (int)max((int64_t)0, min((int64_t)8, c.d - col));
    if (c.dx)
        store8<E>((typename E::raw *)c.dx + t * c.lddx, col, n, v);
    if (c.ds)
        store8<S>((typename S::raw *)c.ds + t * c.ldds, col, n, v);
}

// grid: groups of G threads, each walks over rows g, g + groups, ... and leaves the sums of
// its columns in partial[g].
template <class E, class S, int G, int NC, bool FULL>
__global__ __launch_bounds__(G > 256 ? G : 256) void k_norm_back(NormCall c, int groups)
{
    __shared__ double sh[16];
    constexpr int B = G > 256 ? G : 256;
    const int g = blockIdx.x * (B / G) + threadIdx.x / G, i = threadIdx.x % G;
    if (g >= groups)
        return;
    float dw[NC][8], w[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        weight8_of<E>(c, (int64_t)(k * G + i) * 8, w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[k][j] = 0.f;
    }
    for (int64_t t = g; t < c.T; t += groups) {
        const typename S::raw *sum = (const typename S::raw *)c.sum + t * c.ldsum;
        const typename E::raw *dy = (const typename E::raw *)c.dy + t * c.lddy;
        const typename S::raw *past = (const typename S::raw *)c.dsum + t * c.lddsum;
        Raw8<S> sr[NC], pr[NC];
        Raw8<E> yr[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int64_t col = (int64_t)(k * G + i) * 8;
            sr[k] = row8<S, FULL>(sum, col, c.d);
            yr[k] = row8<E, FULL>(dy, col, c.d);
        }
        if (c.dsum)
#pragma unroll
            for (int k = 0; k < NC; ++k)
                pr[k] = row8<S, FULL>(past, (int64_t)(k * G + i) * 8, c.d);
        const float rstd = c.rstd[t];
        float h[NC][8], gr[NC][8];
        double m = 0.0;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            widen8<S>(sr[k], h[k]);
            widen8<E>(yr[k], gr[k]);
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[k][j] *= rstd;
                dw[k][j] = fmaf(gr[k][j], h[k][j], dw[k][j]);
                gr[k][j] *= w[k][j];
                part = fmaf(gr[k][j], h[k][j], part);
            }
            m += (double)part;
        }
        const float mean = (float)(row_sum<G>(m, sh) / c.d);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float v[8];
            if (c.dsum) {
                widen8<S>(pr[k], v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += rstd * (gr[k][j] - h[k][j] * mean);
            put_ds<E, S>(c, t, (int64_t)(k * G + i) * 8, v);
        }
    }
    if (c.dweight)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int64_t col = (int64_t)(k * G + i) * 8;
            store8<F32>(c.partial + (int64_t)g * c.d, col, (int)max((int64_t)0, min((int64_t)8, c.d - col)), dw[k]);
        }
}

// Rows of any length: one block per row, sums of columns by a kernel of their own.
template <class E, class S>
__global__ __launch_bounds__(1024) void k_norm_back_wide(NormCall c)
{
    __shared__ double sh[16];
    const int64_t t = block_at();
    if (t >= c.T)
        return;
    const typename S::raw *sum = (const typename S::raw *)c.sum + t * c.ldsum;
    const typename E::raw *dy = (const typename E::raw *)c.dy + t * c.lddy;
    const typename S::raw *past = (const typename S::raw *)c.dsum + t * c.lddsum;
    const int rounds = (c.d + 8 * 1024 - 1) / (8 * 1024);
    const float rstd = c.rstd[t];
    double m = 0.0;
    for (int k = 0; k < rounds; ++k) {
        const int64_t col = ((int64_t)k * 1024 + threadIdx.x) * 8;
        float h[8], g[8], w[8], part = 0.f;
        widen8<S>(row8<S, false>(sum, col, c.d), h);
        widen8<E>(row8<E, false>(dy, col, c.d), g);
        weight8_of<E>(c, col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            part = fmaf(g[j] * w[j], h[j] * rstd, part);
        m += (double)part;
    }
    const float mean = (float)(row_sum<1024>(m, sh) / c.d);
    for (int k = 0; k < rounds; ++k) {
        const int64_t col = ((int64_t)k * 1024 + threadIdx.x) * 8;
        float h[8], g[8], w[8], v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        widen8<S>(row8<S, false>(sum, col, c.d), h);
        widen8<E>(row8<E, false>(dy, col, c.d), g);
        if (c.dsum)
            widen8<S>(row8<S, false>(past, col, c.d), v);
        weight8_of<E>(c, col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] += rstd * (g[j] * w[j] - h[j] * rstd * mean);
        put_ds<E, S>(c, t, col, v);
    }
}

// Column sums of long rows: a wave of 64 columns, rows part, part + parts, ...
template <class E, class S>
__global__ __launch_bounds__(64) void k_norm_cols(NormCall c, int parts)
{
    const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (col >= c.d)
        return;
    float dw = 0.f;
    for (int64_t t = blockIdx.y; t < c.T; t += parts)
        dw = fmaf(E::to_f(((const typename E::raw *)c.dy)[t * c.lddy + col]),
                  S::to_f(((const typename S::raw *)c.sum)[t * c.ldsum + col]) * c.rstd[t], dw);
    c.partial[(int64_t)blockIdx.y * c.d + col] = dw;
}

// dweight[i] = sum over the rows of partial, sixteen lanes of rows joined in LDS
__global__ __launch_bounds__(1024) void k_norm_join(NormCall c, int parts)
{
    __shared__ float sh[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.f;
    if (col < c.d)
#pragma unroll 16
        for (int p = w; p < parts; p += 16)
            v += c.partial[(int64_t)p * c.d + col];
    sh[w][lane] = v;
    __syncthreads();
    if (w || col >= c.d)
        return;
#pragma unroll
    for (int q = 1; q < 16; ++q)
        v += sh[q][lane];
    store_el(c.dweight, col, v, c.grad_dtype);
}

template <class E, class S, bool FULL>
void forward_of(const NormCall &c, const NormPlan &p, hipStream_t st)
{
    if constexpr (FULL) {
        if (p.chunks == 0) {  // (long rows have one kernel)
            forward_of<E, S, false>(c, p, st);
            return;
        }
    } else if (p.chunks == 0) {
        hipLaunchKernelGGL((k_norm_wide<E, S>), dim_of(block_grid(c.T)), dim3(1024), 0, st, c);
        return;
    }
#define ECF_NORM(G, NC)                                                                                         \
    hipLaunchKernelGGL((k_norm<E, S, G, NC, FULL>),                                                             \
                       dim_of(block_grid((c.T + (G < 256 ? 256 / G : 1) - 1) / (G < 256 ? 256 / G : 1))),       \
                       dim3(G > 256 ? G : 256), 0, st, c)
    if (p.group == 64 && p.chunks == 1)
        ECF_NORM(64, 1);
    else if (p.group == 64)
        ECF_NORM(64, 2);
    else if (p.group == 256 && p.chunks == 1)
        ECF_NORM(256, 1);
    else if (p.group == 256 && p.chunks == 2)
        ECF_NORM(256, 2);
    else if (p.group == 256)
        ECF_NORM(256, 4);
    else
        ECF_NORM(1024, 2);
#undef ECF_NORM
}

template <class E, class S, bool FULL>
void backward_of(const NormCall &c, const NormPlan &p, int parts, hipStream_t st)
{
    if constexpr (FULL) {
        if (p.chunks == 0) {
            backward_of<E, S, false>(c, p, parts, st);
            return;
        }
    } else if (p.chunks == 0) {
        if (c.dx || c.ds)
            hipLaunchKernelGGL((k_norm_back_wide<E, S>), dim_of(block_grid(c.T)), dim3(1024), 0, st, c);
        if (c.dweight)
            hipLaunchKernelGGL((k_norm_cols<E, S>), dim3((c.d + 63) / 64, parts), dim3(64), 0, st, c, parts);
        return;
    }
#define ECF_NORM(G, NC)                                                                                          \
    hipLaunchKernelGGL((k_norm_back<E, S, G, NC, FULL>), dim3((parts + (G < 256 ? 256 / G : 1) - 1) / (G < 256 ? 256 / G : 1)), \
                       dim3(G > 256 ? G : 256), 0, st, c, parts)
    if (p.group == 64 && p.chunks == 1)
        ECF_NORM(64, 1);
    else if (p.group == 64)
        ECF_NORM(64, 2);
    else if (p.group == 256 && p.chunks == 1)
        ECF_NORM(256, 1);
    else if (p.group == 256 && p.chunks == 2)
        ECF_NORM(256, 2);
    else if (p.group == 256)
        ECF_NORM(256, 4);
    else
        ECF_NORM(1024, 2);
#undef ECF_NORM
}

}  // namespace

int launch_norm_forward(const NormCall &c, hipStream_t st)
{
    ProfScope prof("norm", st);
    const NormPlan p = norm_plan(c.d);
    with_pair(c.dtype, c.sum_dtype, [&](auto e, auto s) {
        using E = decltype(e);
        using S = decltype(s);
        if (c.d % 8 == 0)
            forward_of<E, S, true>(c, p, st);
        else
            forward_of<E, S, false>(c, p, st);
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_norm_backward(const NormCall &c, hipStream_t st)
{
    ProfScope prof("norm_backward", st);
    const int parts = norm_partial_rows(c.T, c.d);
    if (c.T > 0 && (c.dx || c.ds || c.dweight)) {
        const NormPlan p = norm_plan(c.d);
        with_pair(c.dtype, c.sum_dtype, [&](auto e, auto s) {
            using E = decltype(e);
            using S = decltype(s);
            if (c.d % 8 == 0)
                backward_of<E, S, true>(c, p, parts, st);
            else
                backward_of<E, S, false>(c, p, parts, st);
        });
        ECF_HIP_CHECK(hipGetLastError());
    }
    if (c.dweight) {
        hipLaunchKernelGGL(k_norm_join, dim3((c.d + 63) / 64), dim3(1024), 0, st, c, parts);
        ECF_HIP_CHECK(hipGetLastError());
    }
    return ECF_OK;
}

}  // namespace ecf
