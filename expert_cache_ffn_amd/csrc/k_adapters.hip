// Low-rank adapters of many requests beside a shared projection:
//   out[t] = residual[t] + scale[a] * B[a] (A[a] x[t]),  a the token's adapter,
// and the gradients.  Three products, in two layouts of the adapters' matrices each:
//   shrink  h[t][j] = sum_k x[t][k] M(j, k)          forward A, backward B's transpose
//   expand  out[t][i] = res[t][i] + sum_j h[t][j] M(i, j)   forward B, backward A's transpose
//   outer   d(j, i) = sum_t g[t][j] x[t][i]          dA, dB
// The tokens come sorted by adapter; a block has a tile of up to 64 of one adapter's
// (shrink, expand) or walks over the adapters in a run of the order (outer), so one launch
// serves all requests.  Few tokens need no order: each is a block of its own.
//
// x, the residual and the output are read and written once, which bounds all of them; the
// matrices are shared by 64 tokens (by a run of them).
//
// What lies between shrink and expand (h, in the backward pass g) stays in fp32.  As an operand
// of a bf16 product it is split into two bf16 parts (16 bits in all; three parts, so all 24
// bits, where the output is fp32); fp16 and fp32 take fp32 products there, whose rate the
// memory still hides at ranks up to 32.
#include "tokens_device.h"

namespace ecf {
namespace {

typedef float f32x4a __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

constexpr int kKC = 128;   // k per staged chunk of a shrink
constexpr int kRC = 64;    // most ranks at a time
constexpr int kCols = 256; // columns per block of an expand
constexpr int kOuterCols = 128;

struct Tile {
    int a, row0, rows;  // adapter (n: none), first row and rows of the order; rows 0: no tile
};

// The tile's adapter: the last whose first tile is not behind it.
__device__ __forceinline__ Tile tile_of(const AdapterOrder &o, int b)
{
    const int lane = threadIdx.x & 63;
    if (b >= o.tiles[o.n + 1])
        return {0, 0, 0};
    int a = -1;
    for (int e0 = 0; e0 <= o.n; e0 += 64)
        a += __popcll(__ballot(e0 + lane <= o.n && o.tiles[min(e0 + lane, o.n)] <= b));
    const int row0 = o.offsets[a] + (b - o.tiles[a]) * kTileRows;
    const int end = a < o.n ? o.offsets[a + 1] : o.T;
    return {a, row0, min(kTileRows, end - row0)};
}

// The adapter of row `row` of the order (one with an adapter): the last that begins at or
// before it.
__device__ __forceinline__ int adapter_of(const AdapterOrder &o, int row)
{
    const int lane = threadIdx.x & 63;
    int a = -1;
    for (int e0 = 0; e0 < o.n; e0 += 64)
        a += __popcll(__ballot(e0 + lane < o.n && o.offsets[min(e0 + lane, o.n)] <= row));
    return a;
}

__device__ __forceinline__ float scale_of(const float *scale, int a) { return scale ? scale[a] : 1.f; }

// v as a sum of bf16 values, the k-th of them
__device__ __forceinline__ uint16_t bf16_part(float &left)
{
    const uint16_t p = BF16::from_f(left);
    left -= BF16::to_f(p);
    return p;
}

__device__ __forceinline__ f32x4a mfma_bf16(u32x4_t a, u32x4_t b, f32x4a c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// c(j, t) += sum over 32 k of m(j, k) x(t, k): a lane holds k = 8 (lane / 16) .. + 7 of row lane % 16
template <class E, class X>
__device__ __forceinline__ f32x4a product32(const Raw8<E> &m, const Raw8<X> &x, f32x4a c)
{
    if constexpr (std::is_same<E, X>::value && std::is_same<E, BF16>::value) {
        return mfma_bf16(m.v[0], x.v[0], c);
    } else if constexpr (std::is_same<E, X>::value && std::is_same<E, F16>::value) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, m.v[0]), __builtin_bit_cast(half8_t, x.v[0]), c, 0,
                                                      0, 0);
    } else if constexpr (std::is_same<E, BF16>::value) {  // fp32 in three parts
        float v[8];
        widen8<X>(x, v);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            u32x4_t b;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t lo = bf16_part(v[2 * q]), hi = bf16_part(v[2 * q + 1]);
                b[q] = lo | hi << 16;
            }
            c = mfma_bf16(m.v[0], b, c);
        }
        return c;
    } else {
        float a[8], b[8];
        widen8<E>(m, a);
        widen8<X>(x, b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
}

// ---- shrink ----------------------------------------------------------------------------
// grid: tiles, splits of K, chunks of 64 ranks.  A wave has 16 tokens, all ranks of the chunk.
// A chunk of M goes through LDS as [rank][k], zeros past its ends.
template <class E, class X, bool OF_B, int NJ, bool FULL>
__global__ __launch_bounds__(256) void k_shrink(ShrinkCall c)
{
    typedef typename E::raw raw;
    constexpr int RP = NJ * 16, PITCH = kKC + 16 / sizeof(raw);
    __shared__ __align__(16) raw lds[RP * PITCH];
    const Tile tl = tile_of(c.o, blockIdx.x);
    if (tl.rows <= 0 || tl.a >= c.o.n)
        return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r15 = lane & 15, kg = lane >> 4;
    const int j0 = blockIdx.z * kRC, k0 = blockIdx.y * c.split_k, k1 = min(c.K, k0 + c.split_k);
    const raw *m = (const raw *)c.m + (int64_t)tl.a * c.r * c.K;
    const int token = c.o.order[tl.row0 + min(w * 16 + r15, tl.rows - 1)];
    const typename X::raw *x = (const typename X::raw *)c.x + (int64_t)token * c.ldx;
    const bool on = w * 16 < tl.rows;
    f32x4a acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        acc[j] = f32x4a{0.f, 0.f, 0.f, 0.f};
    for (int kc = k0; kc < k1; kc += kKC) {
        Raw8<X> xr[4];
        if (on)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                xr[s] = row8<X, FULL>(x, kc + s * 32 + kg * 8, c.K);
        __syncthreads();  // the chunk before is read
        if constexpr (!OF_B) {
            for (int i = tid; i < RP * (kKC / 8); i += 256) {
                const int j = i / (kKC / 8), k = i % (kKC / 8) * 8;
                Raw8<E> v = row8<E, FULL>(m + (int64_t)min(j0 + j, c.r - 1) * c.K, kc + k, c.K);
                if (j0 + j >= c.r)
                    v = Raw8<E>{};
                *(Raw8<E> *)(lds + j * PITCH + k) = v;
            }
        } else {
            // rows of r ranks, one for each k
            const int nj = min(RP, c.r - j0);
            for (int i = tid; i < kKC * (RP / 8); i += 256) {
                const int k = i / (RP / 8), j = i % (RP / 8) * 8;
                Raw8<E> v{};
                if (kc + k < c.K && j < nj)
                    v = row8<E, false>(m + (int64_t)(kc + k) * c.r + j0, j, nj);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (sizeof(raw) == 2)
                        lds[(j + e) * PITCH + k] = (uint16_t)(v.v[0][e >> 1] >> (16 * (e & 1)));
                    else
                        lds[(j + e) * PITCH + k] = __uint_as_float(v.v[e >> 2][e & 3]);
                }
            }
        }
        __syncthreads();
        if (on)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const Raw8<E> mr = *(const Raw8<E> *)(lds + (j * 16 + r15) * PITCH + s * 32 + kg * 8);
                    acc[j] = product32<E, X>(mr, xr[s], acc[j]);
                }
    }
    if (w * 16 + r15 < tl.rows) {
        float *out = c.part + ((int64_t)blockIdx.y * c.o.T + token) * c.r + j0;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + j * 16 + kg * 4 + e < c.r)
                    out[j * 16 + kg * 4 + e] = acc[j][e];
    }
}

// ---- expand ----------------------------------------------------------------------------
// grid: tiles, slices of 256 columns.  A wave has 64 columns and the tile's 64 tokens.  Row m of
// MFMA i is column 16 (m / 4) + 4 i + m % 4, so that a lane's four MFMAs leave it 16 columns
// in a row of one token.
template <class E, class O, bool OF_A, bool FULL>
__global__ __launch_bounds__(256) void k_expand(ExpandCall c)
{
    typedef typename E::raw raw;
    constexpr bool BF = std::is_same<E, BF16>::value;
    constexpr int PARTS = !BF ? 1 : std::is_same<O, F32>::value ? 3 : 2;
    constexpr int PITCH = kRC + 16 / sizeof(raw);
    constexpr int HP = BF ? (PARTS * kRC + 31) / 32 * 32 + 8 : kRC + 4;  // of h's rows, in bf16 or fp32
    typedef typename std::conditional<BF, uint16_t, float>::type hraw;
    __shared__ __align__(16) raw ml[kCols * PITCH];
    __shared__ __align__(16) hraw hl[kTileRows * HP];
    const Tile tl = tile_of(c.o, blockIdx.x);
    if (tl.rows <= 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r15 = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.y * kCols;
    const bool none = tl.a >= c.o.n;  // the tokens without an adapter
    const int a = none ? 0 : tl.a;
    const float scale = none ? 0.f : scale_of(c.scale, a);
    const raw *m = (const raw *)c.m + (int64_t)a * c.r * c.N;
    const int col = n0 + w * 64 + kg * 16;
    int token[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
        token[b] = c.o.order[tl.row0 + min(b * 16 + r15, tl.rows - 1)];
    Raw8<O> res[4][2];
    if (c.residual && c.out)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                res[b][q] = row8<O, FULL>((const typename O::raw *)c.residual + token[b] * c.ldres, col + 8 * q, c.N);
    f32x4a acc[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[b][i] = f32x4a{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < c.r; j0 += kRC) {
        const int nj = min(kRC, c.r - j0), rp = (nj + 15) / 16 * 16;
        __syncthreads();  // the ranks before are read
        // h of the tile's tokens: the splits' sum, written out once
        for (int i = tid; i < kTileRows * rp; i += 256) {
            const int row = i / rp, j = i % rp;
            float v = 0.f;
            if (row < tl.rows && j < nj) {
                const int t = c.o.order[tl.row0 + row];
                if (!none)
                    for (int s = 0; s < c.splits; ++s)
                        v += c.part[((int64_t)s * c.o.T + t) * c.r + j0 + j];
                if (c.h && blockIdx.y == 0)
                    c.h[(int64_t)t * c.r + j0 + j] = c.scaled ? v * scale : v;
                v *= scale;
            }
            if constexpr (BF) {
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    hl[row * HP + p * rp + j] = bf16_part(v);
            } else {
                hl[row * HP + j] = v;
            }
        }
        if (none || !c.out)
            continue;
        if constexpr (BF) {  // the parts end in a whole step of 32
            const int slots = PARTS * rp, more = (32 - slots % 32) % 32;
            for (int i = tid; i < kTileRows * more; i += 256)
                hl[i / more * HP + slots + i % more] = 0;
        }
        if constexpr (!OF_A) {
            for (int i = tid; i < kCols * (rp / 8); i += 256) {
                const int n = i / (rp / 8), j = i % (rp / 8) * 8;
                Raw8<E> v{};
                if (n0 + n < c.N && j < nj)
                    v = row8<E, false>(m + (int64_t)(n0 + n) * c.r + j0, j, nj);
                *(Raw8<E> *)(ml + n * PITCH + j) = v;
            }
        } else {
            for (int i = tid; i < rp * (kCols / 8); i += 256) {
                const int j = i / (kCols / 8), n = i % (kCols / 8) * 8;
                Raw8<E> v{};
                if (j < nj)
                    v = row8<E, FULL>(m + (int64_t)(j0 + j) * c.N, n0 + n, c.N);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (sizeof(raw) == 2)
                        ml[(n + e) * PITCH + j] = (uint16_t)(v.v[0][e >> 1] >> (16 * (e & 1)));
                    else
                        ml[(n + e) * PITCH + j] = __uint_as_float(v.v[e >> 2][e & 3]);
                }
            }
        }
        __syncthreads();
        if constexpr (BF) {
            const int slots = PARTS * rp;
            int j = kg * 8;
            for (int s = 0; s < slots; s += 32, j += 32) {
                while (j >= rp)
                    j -= rp;
                u32x4_t mf[4], hf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mf[i] = *(const u32x4_t *)(ml + (w * 64 + 16 * (r15 >> 2) + 4 * i + (r15 & 3)) * PITCH + j);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    hf[b] = *(const u32x4_t *)(hl + (b * 16 + r15) * HP + s + kg * 8);
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[b][i] = mfma_bf16(mf[i], hf[b], acc[b][i]);
            }
        } else {
            for (int s = 0; s < rp; s += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float mv = E::to_f(ml[(w * 64 + 16 * (r15 >> 2) + 4 * i + (r15 & 3)) * PITCH + s + kg]);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(mv, hl[(b * 16 + r15) * HP + s + kg], acc[b][i], 0, 0, 0);
                }
        }
    }
    if (!c.out)
        return;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b * 16 + r15 >= tl.rows)
            continue;
        typename O::raw *out = (typename O::raw *)c.out + token[b] * c.ldout;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c.residual)
                widen8<O>(res[b][q], v);
            if (!none)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += acc[b][2 * q + (e >> 2)][e & 3];
            store8<O>(out, col + 8 * q, max(0, min(8, c.N - col - 8 * q)), v);
        }
    }
}

// ---- few tokens ------------------------------------------------------------------------
// token t's adapter, -1: none
__device__ __forceinline__ int adapter_at(const AdapterOrder &o, int t)
{
    const int64_t a = o.wide ? ((const int64_t *)o.idx)[t] : ((const int32_t *)o.idx)[t];
    return a >= 0 && a < o.n ? (int)a : -1;
}

// grid: ranks, tokens; the four waves share K
template <class E, bool FULL>
__global__ __launch_bounds__(256) void k_few_shrink(ShrinkCall c)
{
    __shared__ float sh[4];
    const int j = blockIdx.x, t = blockIdx.y, tid = threadIdx.x;
    const int a = adapter_at(c.o, t);
    float s = 0.f;
    if (a >= 0) {
        const typename E::raw *m = (const typename E::raw *)c.m + ((int64_t)a * c.r + j) * c.K;
        const typename E::raw *x = (const typename E::raw *)c.x + (int64_t)t * c.ldx;
#pragma unroll 4
        for (int k = tid * 8; k < c.K; k += 256 * 8) {
            float u[8], v[8];
            const Raw8<E> mr = row8<E, FULL>(m, k, c.K), xr = row8<E, FULL>(x, k, c.K);
            widen8<E>(mr, u);
            widen8<E>(xr, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(u[i], v[i], s);
        }
    }
    s = wave_sum_f32(s);
    if ((tid & 63) == 0)
        sh[tid >> 6] = s;
    __syncthreads();
    if (tid == 0)
        c.part[(int64_t)t * c.r + j] = (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

// grid: slices of 64 columns, tokens; a lane has a column
template <class E, class O>
__global__ __launch_bounds__(64) void k_few_expand(ExpandCall c)
{
    __shared__ float h[256];
    const int t = blockIdx.y, lane = threadIdx.x, n = blockIdx.x * 64 + lane;
    const int a = adapter_at(c.o, t);
    const bool none = a < 0;
    const float scale = none ? 0.f : scale_of(c.scale, a);
    for (int j = lane; j < c.r; j += 64) {
        const float v = c.part[(int64_t)t * c.r + j];
        h[j] = v;
        if (c.h && blockIdx.x == 0)
            c.h[(int64_t)t * c.r + j] = v;
    }
    __syncthreads();
    if (n >= c.N)
        return;
    float s = 0.f;
    if (!none) {
        const typename E::raw *m = (const typename E::raw *)c.m + ((int64_t)a * c.N + n) * c.r;
#pragma unroll 2
        for (int j = 0; j < c.r; j += 8) {
            float u[8];
            widen8<E>(row8<E, false>(m, j, c.r), u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(u[i], j + i < c.r ? h[j + i] : 0.f, s);
        }
    }
    float y = scale * s;
    if (none)
        y = 0.f;
    if (c.residual)
        y = O::to_f(((const typename O::raw *)c.residual)[t * c.ldres + n]) + y;
    ((typename O::raw *)c.out)[t * c.ldout + n] = O::from_f(y);
}

// ---- outer -----------------------------------------------------------------------------
// grid: slices of 128 columns, runs of the sorted rows, chunks of 64 ranks.  In each
// adapter's part of the run the four waves take 32 tokens in turn and their sums meet in
// LDS.  An adapter whose tokens all lie in the run is done; the sums of one that goes on in other runs
// are left in the run's slot 0 (it began in an earlier one) or 1 and added by k_outer_join.
// A lane has column 8 (lane % 16) + e of the slice in MFMA e and reads 8 columns of 8 tokens.
template <class X, int NJ, int PARTS, bool FULL>
__global__ __launch_bounds__(256) void k_outer(OuterCall c, int per)
{
    constexpr bool BF = std::is_same<X, BF16>::value;
    constexpr int RP = NJ * 16, PITCH = kOuterCols + 4;
    __shared__ float sums[RP * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r15 = lane & 15, kg = lane >> 4;
    const int c0 = blockIdx.x * kOuterCols, j0 = blockIdx.z * kRC;
    const int rows = c.o.offsets[c.o.n], beg = blockIdx.y * per, end = min(rows, beg + per);
    if (beg >= end)
        return;
    for (int s0 = beg, s1; s0 < end; s0 = s1) {
        const int a = adapter_of(c.o, s0), o0 = c.o.offsets[a], o1 = c.o.offsets[a + 1];
        s1 = min(o1, end);
        f32x4a acc[NJ][8];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[j][e] = f32x4a{0.f, 0.f, 0.f, 0.f};
        const float gs = scale_of(c.gscale, a);
        for (int t0 = s0 + w * 32; t0 < s1; t0 += 4 * 32) {
            Raw8<X> xr[8];
            float g[NJ][8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int row = t0 + 8 * kg + u;
                const int t = c.o.order[min(row, s1 - 1)];
                xr[u] = row8<X, FULL>((const typename X::raw *)c.x + (int64_t)t * c.ldx, c0 + 8 * r15, c.W);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int at = j0 + j * 16 + r15;
                    const float v = c.g[(int64_t)t * c.r + min(at, c.r - 1)];
                    g[j][u] = at < c.r && row < s1 ? v * gs : 0.f;
                }
                if (row >= s1)
                    xr[u] = Raw8<X>{};
            }
            if constexpr (BF) {
                u32x4_t gp[NJ][PARTS];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t lo = bf16_part(g[j][2 * q]), hi = bf16_part(g[j][2 * q + 1]);
                            gp[j][p][q] = lo | hi << 16;
                        }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // column e of the eight tokens
                    u32x4_t b;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        b[q] = __builtin_amdgcn_perm(xr[2 * q + 1].v[0][e >> 1], xr[2 * q].v[0][e >> 1],
                                                     e & 1 ? 0x07060302 : 0x05040100);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
                            acc[j][e] = mfma_bf16(gp[j][p], b, acc[j][e]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    float v[8];
                    widen8<X>(xr[u], v);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[j][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(g[j][u], v[e], acc[j][e], 0, 0, 0);
                }
            }
        }
        for (int q = 0; q < 4; ++q) {
            if (w == q)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float *s = sums + (j * 16 + kg * 4 + i) * PITCH + 8 * r15 + e;
                            *s = q ? *s + acc[j][e][i] : acc[j][e][i];
                        }
            __syncthreads();
        }
        const bool whole = o0 >= beg && o1 <= end;
        float *slot = c.slots + ((int64_t)blockIdx.y * 2 + (o0 >= beg)) * c.r * c.W;
        for (int i = tid; i < RP * kOuterCols; i += 256) {
            // along the side that is contiguous
            const int j = c.of_b ? i % RP : i / kOuterCols, x = c.of_b ? i / RP : i % kOuterCols;
            if (j0 + j >= c.r || c0 + x >= c.W)
                continue;
            const float v = sums[j * PITCH + x];
            const int64_t at = c.of_b ? (int64_t)(c0 + x) * c.r + j0 + j : (int64_t)(j0 + j) * c.W + c0 + x;
            if (whole)
                store_el(c.d, (int64_t)a * c.r * c.W + at, v, c.grad_dtype);
            else
                slot[at] = v;
        }
        __syncthreads();
    }
}

// grid: blocks of 1024 elements, adapters
__global__ __launch_bounds__(256) void k_outer_join(OuterCall c, int per)
{
    const int a = blockIdx.y;
    const int o0 = c.o.offsets[a], o1 = c.o.offsets[a + 1];
    const int first = o0 / per, last = (o1 - 1) / per;
    if (o1 > o0 && first == last)
        return;
    const int64_t size = (int64_t)c.r * c.W;
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < min(size, ((int64_t)blockIdx.x + 1) * 1024); i += 256) {
        float v = 0.f;
        if (o1 > o0)
            for (int q = first; q <= last; ++q)
                v += c.slots[((int64_t)q * 2 + (q == first)) * size + i];
        store_el(c.d, (int64_t)a * size + i, v, c.grad_dtype);
    }
}

// ---- launches --------------------------------------------------------------------------

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

int most_tiles(const AdapterOrder &o) { return o.T / kTileRows + (o.n + 1 < o.T ? o.n + 1 : o.T); }
int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

template <class E, class X, bool OF_B, bool FULL>
void shrink_of(const ShrinkCall &c, hipStream_t st)
{
    const dim3 grid(most_tiles(c.o), c.splits, (c.r + kRC - 1) / kRC);
    switch (rank_blocks(c.r)) {
    case 1: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 1, FULL>), grid, dim3(256), 0, st, c); break;
    case 2: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 2, FULL>), grid, dim3(256), 0, st, c); break;
    default: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 4, FULL>), grid, dim3(256), 0, st, c);
    }
}

template <class X, int PARTS, bool FULL>
void outer_of(const OuterCall &c, int per, hipStream_t st)
{
    const dim3 grid((c.W + kOuterCols - 1) / kOuterCols, c.chunks, (c.r + kRC - 1) / kRC);
    switch (rank_blocks(c.r)) {
    case 1: hipLaunchKernelGGL((k_outer<X, 1, PARTS, FULL>), grid, dim3(256), 0, st, c, per); break;
    case 2: hipLaunchKernelGGL((k_outer<X, 2, PARTS, FULL>), grid, dim3(256), 0, st, c, per); break;
    default: hipLaunchKernelGGL((k_outer<X, 4, PARTS, FULL>), grid, dim3(256), 0, st, c, per);
    }
}

}  // namespace

// Splits of K: two blocks a CU where there are few tiles, 256 of K each at least, at most 8
// (each adds a part of h that every block of the expand reads).
int shrink_splits(int T, int K)
{
    int s = kShrinkBlocks / (T / kTileRows + 1);
    s = s < kShrinkSplits ? s : kShrinkSplits;
    const int most = (K + 255) / 256;
    s = s < most ? s : most;
    return s > 1 ? s : 1;
}

int launch_shrink(const ShrinkCall &c, hipStream_t st)
{
    ProfScope prof("adapter_shrink", st);
    with_bool(c.K % 8 == 0, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (c.of_b)
            with_pair(c.dtype, c.x_dtype, [&](auto e, auto x) { shrink_of<decltype(e), decltype(x), true, FULL>(c, st); });
        else
            with_element(c.dtype, [&](auto e) { shrink_of<decltype(e), decltype(e), false, FULL>(c, st); });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_expand(const ExpandCall &c, hipStream_t st)
{
    ProfScope prof("adapter_expand", st);
    const dim3 grid(most_tiles(c.o), c.out ? (c.N + kCols - 1) / kCols : 1);
    with_bool(c.N % 8 == 0, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (c.of_a)
            with_element(c.dtype, [&](auto e) {
                hipLaunchKernelGGL((k_expand<decltype(e), decltype(e), true, FULL>), grid, dim3(256), 0, st, c);
            });
        else
            with_pair(c.dtype, c.out_dtype, [&](auto e, auto o) {
                hipLaunchKernelGGL((k_expand<decltype(e), decltype(o), false, FULL>), grid, dim3(256), 0, st, c);
            });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_few_shrink(const ShrinkCall &c, hipStream_t st)
{
    ProfScope prof("adapter_few_shrink", st);
    with_element(c.dtype, [&](auto e) {
        using E = decltype(e);
        if (c.K % 8 == 0)
            hipLaunchKernelGGL((k_few_shrink<E, true>), dim3(c.r, c.o.T), dim3(256), 0, st, c);
        else
            hipLaunchKernelGGL((k_few_shrink<E, false>), dim3(c.r, c.o.T), dim3(256), 0, st, c);
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_few_expand(const ExpandCall &c, hipStream_t st)
{
    ProfScope prof("adapter_few_expand", st);
    with_pair(c.dtype, c.out_dtype, [&](auto e, auto o) {
        hipLaunchKernelGGL((k_few_expand<decltype(e), decltype(o)>), dim3((c.N + 63) / 64, c.o.T), dim3(64), 0, st, c);
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

// Runs of the sorted rows: two blocks a CU over all slices, 128 rows each at least.
int outer_chunks(int T, int W)
{
    const int slices = (W + kOuterCols - 1) / kOuterCols, most = (T + 127) / 128;
    const int s = 512 / slices;
    return s < 1 || most < 1 ? 1 : s < most ? s : most;
}

int launch_outer(const OuterCall &c, hipStream_t st)
{
    ProfScope prof("adapter_outer", st);
    const int per = c.o.T > 0 ? ((c.o.T + c.chunks - 1) / c.chunks + 31) / 32 * 32 : 32;
    with_bool(c.W % 8 == 0, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (c.x_dtype == ECF_BF16) {
            if (c.grad_dtype == ECF_F32)
                outer_of<BF16, 3, FULL>(c, per, st);
            else
                outer_of<BF16, 2, FULL>(c, per, st);
        } else if (c.x_dtype == ECF_F32) {
            outer_of<F32, 1, FULL>(c, per, st);
        } else {
            outer_of<F16, 1, FULL>(c, per, st);
        }
    });
    ECF_HIP_CHECK(hipGetLastError());
    const int64_t size = (int64_t)c.r * c.W;
    hipLaunchKernelGGL(k_outer_join, dim3((unsigned)((size + 1023) / 1024), c.o.n), dim3(256), 0, st, c, per);
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

}  // namespace ecf
