// Dense operators for few tokens (at most 64): x W^T, gated or not, as a streaming
// read of the weights: every weight byte is read once, straight into MFMA operand
// registers.
//
// A 16x16 MFMA takes 16 weight rows and 16 tokens at the same k.  With few rows
// per block the 16 rows become RT weight rows at P = 16 / RT places of K, and the
// 16 columns RT tokens at the same P places; the P diagonal RT x RT corners of the
// result are P partial sums (what lies off the diagonal is never looked at).  So a
// block owns RT = 4, 8 or 16 weight rows (of each projection), a load instruction
// reads 256, 128 or 64 consecutive bytes of each row, and a layer of
// 1024 columns still fills 256 CUs.  More than RT tokens take TG groups of RT,
// which share each weight fragment.
//
// The waves of a block share K; their partial sums meet in LDS and are added in a
// fixed order by one thread per output, which applies the epilogue.
//
// Bound by what a CU takes in of weights and x together.  2 x 1024 rows of K 4096, bf16
// (16.8 MB): one token 5.0 to 5.4 us, 16 tokens 8.0 to 9.2; 2.5 us of it are launch and
// first loads, then a CU takes in 38 KB/us (9.7 TB/s of all, the weights lying in the
// memory-side cache).  x is read anew for every 16 rows at most, as many bytes as the
// weights at 9 to 16 tokens, so wide layers stay far from the memory's rate: 16 x 4096 to
// 16384 in bf16 41 us (134 MB, 3.3 TB/s), 11 x 7469 to 12864 in fp32 165 us (384 MB, 2.3).
#include "dense_device.h"

namespace ecf {
namespace {

typedef float f32x4a __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

// 16 bytes of A and B per lane into a 16 x 16 tile: 8 k per lane (16-bit types) or
// 4 (fp32, four exact fp32 MFMAs); lanes 16 g .. 16 g + 15 hold k group g.
template <class E>
__device__ __forceinline__ f32x4a mfma_chunk(u32x4_t a, u32x4_t b, f32x4a c)
{
    if constexpr (std::is_same<E, BF16>::value) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    } else if constexpr (std::is_same<E, F16>::value) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c,
                                                      0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
        return c;
    }
}

template <class E>
__device__ __forceinline__ u32x4_t load_chunk(const typename E::raw *p)
{
    if constexpr (sizeof(typename E::raw) == 2)
        return ((const any128x2 *)p)->v;
    else
        return __builtin_bit_cast(u32x4_t, ((const any128x4 *)p)->v);
}

// Chunk `ch` (16 bytes) of a row of K elements, zeros past its end.
template <class E>
__device__ __forceinline__ u32x4_t chunk_of(const void *row, int ch, int K)
{
    constexpr int EPC = 16 / sizeof(typename E::raw);
    const typename E::raw *p = (const typename E::raw *)row + (int64_t)ch * EPC;
    const int n = K - ch * EPC;
    if (n >= EPC) {
        if constexpr (EPC == 8)
            return ((const any128x2 *)p)->v;
        else
            return __builtin_bit_cast(u32x4_t, ((const any128x4 *)p)->v);
    }
    u32x4_t v = {0, 0, 0, 0};
    if (n <= 0)
        return v;
    if (K >= EPC) {  // the row's last 16 bytes, moved down
        const int s = EPC - n;
        if constexpr (EPC == 8)
            return shift_down16(((const any128x2 *)(p - s))->v, s);
        v = __builtin_bit_cast(u32x4_t, ((const any128x4 *)(p - s))->v);
        if (s & 2)
            v = u32x4_t{v[2], v[3], 0, 0};
        if (s & 1)
            v = u32x4_t{v[1], v[2], v[3], 0};
        return v;
    }
#pragma unroll
    for (int j = 0; j < EPC; ++j)
        if (j < n) {
            if constexpr (EPC == 8)
                v[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            else
                v[j] = __float_as_uint(p[j]);
        }
    return v;
}

// grid: one block per RT weight rows
template <class E, bool GATED, int RT, int TG>
__global__ __launch_bounds__(64 * kFewWaves) void k_dense_few(DenseGemm g)
{
    constexpr int P = 16 / RT, H = GATED ? 2 : 1, EPC = 16 / sizeof(typename E::raw);
    constexpr int U = 4;  // steps whose loads are under way together
    __shared__ float part[kFewWaves][H][TG][P][RT][RT + 1];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, nw = (int)blockDim.x >> 6;
    const int r = lane & 15, kg = lane >> 4;  // operand row (and column), k group
    const int n0 = (int)blockIdx.x * RT;
    const int wrow = min(n0 + r % RT, g.N - 1);
    const int place = r / RT;
    const typename E::raw *wp[H], *xp[TG];
#pragma unroll
    for (int h = 0; h < H; ++h)
        wp[h] = (const typename E::raw *)g.b[h] + (int64_t)wrow * g.ldb;
#pragma unroll
    for (int t = 0; t < TG; ++t)
        xp[t] = (const typename E::raw *)g.a[0] + (int64_t)min(t * RT + r % RT, g.M - 1) * g.lda;
    // step s: chunks 4 P s .. 4 P (s + 1), this lane's at 4 P s + 4 place + k group
    const int steps = (g.K + EPC * 4 * P - 1) / (EPC * 4 * P);
    const int s0 = (int)((int64_t)steps * w / nw), s1 = (int)((int64_t)steps * (w + 1) / nw);
    f32x4a acc[H][TG];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < TG; ++t)
            acc[h][t] = f32x4a{0.f, 0.f, 0.f, 0.f};
    // Whole steps: every chunk lies inside its row, so no load sits behind a branch
    // (at the branch's end the compiler would wait for it).
    const int whole = min(s1, g.K / (EPC * 4 * P)), at = (place * 4 + kg) * EPC;
    const typename E::raw *wq[H], *xq[TG];
#pragma unroll
    for (int h = 0; h < H; ++h)
        wq[h] = wp[h] + at;
#pragma unroll
    for (int t = 0; t < TG; ++t)
        xq[t] = xp[t] + at;
    auto steps_at = [&](int s, auto n) __attribute__((always_inline)) {
        constexpr int NU = decltype(n)::value;
        u32x4_t wv[NU][H], xv[NU][TG];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int64_t o = (int64_t)(s + u) * (EPC * 4 * P);
#pragma unroll
            for (int h = 0; h < H; ++h)
                wv[u][h] = load_chunk<E>(wq[h] + o);
#pragma unroll
            for (int t = 0; t < TG; ++t)
                xv[u][t] = load_chunk<E>(xq[t] + o);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    acc[h][t] = mfma_chunk<E>(wv[u][h], xv[u][t], acc[h][t]);
    };
    int s = s0;
    for (; s + U <= whole; s += U)
        steps_at(s, std::integral_constant<int, U>{});
    for (; s < whole; ++s)
        steps_at(s, std::integral_constant<int, 1>{});
    if (s < s1) {  // the row's last, partial step
        const int ch = s * 4 * P + place * 4 + kg;
        u32x4_t wv[H], xv[TG];
#pragma unroll
        for (int h = 0; h < H; ++h)
            wv[h] = chunk_of<E>(wp[h], ch, g.K);
#pragma unroll
        for (int t = 0; t < TG; ++t)
            xv[t] = chunk_of<E>(xp[t], ch, g.K);
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int t = 0; t < TG; ++t)
                acc[h][t] = mfma_chunk<E>(wv[h], xv[t], acc[h][t]);
    }
    // a lane holds rows 4 kg .. 4 kg + 3 of column r: keep those whose place is the column's
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = 4 * kg + e;
        if (row / RT == place)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    part[w][h][t][place][row % RT][r % RT] = acc[h][t][e];
    }
    __syncthreads();
    for (int i = tid; i < RT * RT * TG; i += (int)blockDim.x) {
        const int row = i % RT, tok = i / RT, n = n0 + row;
        if (tok >= g.M || n >= g.N)
            continue;
        float z[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float v = 0.f;
            for (int q = 0; q < nw; ++q)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    v += part[q][h][tok / RT][p][row][tok % RT];
            if (g.bias[h])
                v += E::to_f(((const typename E::raw *)g.bias[h])[n]);
            if (g.save[h])
                ((typename E::raw *)g.save[h])[tok * g.ldsave + n] = E::from_f(v);
            z[h] = v;
        }
        if (!g.out[0])
            continue;
        float y = act_value(z[0], g.act);
        if constexpr (GATED)
            y *= z[H - 1];
        const bool f32 = g.out_dtype == ECF_F32;
        if (!GATED && g.res)
            y += f32 ? ((const float *)g.res)[tok * g.ldres + n]
                     : E::to_f(((const typename E::raw *)g.res)[tok * g.ldres + n]);
        if (f32)
            ((float *)g.out[0])[tok * g.ldout + n] = y;
        else
            ((typename E::raw *)g.out[0])[tok * g.ldout + n] = E::from_f(y);
    }
}

template <class E, bool GATED>
void run_few(const DenseGemm &g, const DenseFew &f, hipStream_t st)
{
    const int rt = f.rows, groups = f.groups;
    const dim3 grid((g.N + rt - 1) / rt), block(64 * f.waves);
#define ECF_FEW(R, G) hipLaunchKernelGGL((k_dense_few<E, GATED, R, G>), grid, block, 0, st, g)
    if (rt == 16) {
        if (groups == 1)
            ECF_FEW(16, 1);
        else if (groups == 2)
            ECF_FEW(16, 2);
        else
            ECF_FEW(16, 4);
    } else if (rt == 8) {
        if (groups == 1)
            ECF_FEW(8, 1);
        else if (groups == 2)
            ECF_FEW(8, 2);
        else
            ECF_FEW(8, 4);
    } else {
        if (groups == 1)
            ECF_FEW(4, 1);
        else if (groups == 2)
            ECF_FEW(4, 2);
        else
            ECF_FEW(4, 4);
    }
#undef ECF_FEW
}

}  // namespace

int launch_dense_few(const DenseGemm &g, const DenseFew &f, hipStream_t st)
{
    auto go = [&](auto e) {
        using E = decltype(e);
        if (g.gated)
            run_few<E, true>(g, f, st);
        else
            run_few<E, false>(g, f, st);
    };
    if (g.dtype == ECF_F32)
        go(F32{});
    else if (g.dtype == ECF_BF16)
        go(BF16{});
    else
        go(F16{});
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

}  // namespace ecf
