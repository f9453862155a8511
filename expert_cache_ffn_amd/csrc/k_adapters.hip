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
// matrices are shared by 64 tokens (by a run of them) and come from the caches.  Measured in
// bf16 (a large copy takes 5.0 TB/s): 4096 tokens, 4096 to 4096, rank 16, 8 adapters: shrink
// 12.3 us (2.7 TB/s: few chunks a block behind the chain tiles - order - x), expand 20.8 (3.2:
// all blocks run at once, first all load, then all store); 8192 tokens, 2048 / 4096, rank 32:
// shrink of dout 20 (3.4), expand to dx 21.8 (3.1), both outer products 36.5 (2.8) and 7 for their
// join; 16 tokens of 16 adapters 6.6 us in one kernel.
//
// What lies between shrink and expand (h, in the backward pass g) stays in fp32.  As an operand
// of a bf16 product it is split into three bf16 parts, all its 24 bits, whatever the output's
// type: two parts lose what is left where a residual or another token cancels most of the
// product, and cost about as much.  fp16 and fp32 take fp32 products there, whose rate the
// memory still hides at ranks up to 32.
#include "tokens_device.h"

namespace ecf {
namespace {

typedef float f32x4a __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

constexpr int kKC = kShrinkChunk;
constexpr int kRC = 64;    // most ranks at a time
constexpr int kCols = 512; // columns per block of an expand
constexpr int kParts = 3;  // bf16 values that hold an fp32 one

struct Tile {
    int a, row0, rows;  // adapter (n: none), first row and rows of the order; rows 0: no tile
};

// The tile's adapter is the last whose first tile is not behind it; what is asked of it is loaded
// along with the search, for 64 adapters at a time.
__device__ __forceinline__ Tile tile_of(const AdapterOrder &o, int b)
{
    const int lane = threadIdx.x & 63, last = o.tiles[o.n + 1];
    Tile t{-1, 0, 0};
    for (int e0 = 0; e0 <= o.n; e0 += 64) {
        const int e = min(e0 + lane, o.n);
        const int tile = o.tiles[e], from = o.offsets[e], to = o.offsets[min(e + 1, o.n)];
        const uint64_t before = __ballot(e0 + lane <= o.n && tile <= b);
        if (before == 0)
            break;
        const int i = __popcll(before) - 1;  // (the first tiles never fall)
        t.a = e0 + i;
        t.row0 = __builtin_amdgcn_readlane(from, i) + (b - __builtin_amdgcn_readlane(tile, i)) * kTileRows;
        t.rows = (t.a < o.n ? __builtin_amdgcn_readlane(to, i) : o.T) - t.row0;
    }
    t.rows = b < last ? min(kTileRows, t.rows) : 0;
    return t;
}

__device__ __forceinline__ float scale_of(const float *scale, int a) { return scale ? scale[a] : 1.f; }

// v as a sum of bf16 values, the next of them: its upper half, so that a finite value near fp32's
// largest is not rounded to infinity.  Three hold 24 bits; an infinity is the first and zeros, and what
// is left of a NaN is one, whichever half its bits lie in.
__device__ __forceinline__ uint16_t bf16_part(float &left)
{
    const uint32_t top = __float_as_uint(left) & 0xffff0000u;
    const float p = __uint_as_float(top);
    left = left == p ? 0.f : left - p;
    return (uint16_t)(top >> 16);
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
        for (int p = 0; p < kParts; ++p) {
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
// A chunk of M goes through LDS as [rank][k], zeros past its ends; the loads of the next one
// and of its x are under way over the products of this one.
template <class E, class X, bool OF_B, int NJ, bool FULL, bool RFULL>
struct Shrink {
    typedef typename E::raw raw;
    // per thread: with M as it lies NJ chunks of 8 k of one rank; with its transpose NJ / 2 (1 for 16 ranks, half of
    // the threads) pairs of 8 ranks at two k
    static constexpr int RP = NJ * 16, PITCH = kKC + 16 / sizeof(raw), NP = (NJ + 1) / 2;
    Raw8<X> x[4];
    Raw8<E> m[OF_B ? 2 * NP : NJ];

    __device__ __forceinline__ void load(const ShrinkCall &c, const raw *mat, const typename X::raw *xrow, int j0, int kc, int kg, bool on)
    {
        if (on)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                x[s] = row8<X, FULL>(xrow, kc + s * 32 + kg * 8, c.K);
        const int tid = threadIdx.x;
        if constexpr (!OF_B) {
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const int i = tid + q * 256, j = i / (kKC / 8), k = i % (kKC / 8) * 8;
                m[q] = row8<E, FULL>(mat + (int64_t)min(j0 + j, c.r - 1) * c.K, kc + k, c.K);
                if (j0 + j >= c.r)
                    m[q] = Raw8<E>{};
            }
        } else {
            const int nj = min(RP, c.r - j0);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const int i = tid + q * 256, k = i / (RP / 8) * 2, j = i % (RP / 8) * 8;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m[2 * q + h] = row8<E, RFULL>(mat + (int64_t)min(kc + k + h, c.K - 1) * c.r + j0, j, nj);
                    if (kc + k + h >= c.K)
                        m[2 * q + h] = Raw8<E>{};
                }
            }
        }
    }
    __device__ __forceinline__ void stage(raw *lds) const
    {
        const int tid = threadIdx.x;
        if constexpr (!OF_B) {
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const int i = tid + q * 256;
                *(Raw8<E> *)(lds + i / (kKC / 8) * PITCH + i % (kKC / 8) * 8) = m[q];
            }
        } else {
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const int i = tid + q * 256, k = i / (RP / 8) * 2, j = i % (RP / 8) * 8;
                if (k < kKC)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        raw *at = lds + (j + e) * PITCH + k;
                        if constexpr (sizeof(raw) == 2) {
                            *(uint32_t *)at = __builtin_amdgcn_perm(m[2 * q + 1].v[0][e >> 1], m[2 * q].v[0][e >> 1],
                                                                    e & 1 ? 0x07060302 : 0x05040100);
                        } else {
                            at[0] = __uint_as_float(m[2 * q].v[e >> 2][e & 3]);
                            at[1] = __uint_as_float(m[2 * q + 1].v[e >> 2][e & 3]);
                        }
                    }
            }
        }
    }
};

template <class E, class X, bool OF_B, int NJ, bool FULL, bool RFULL>
__global__ __launch_bounds__(256) void k_shrink(ShrinkCall c)
{
    typedef typename E::raw raw;
    typedef Shrink<E, X, OF_B, NJ, FULL, RFULL> S;
    __shared__ __align__(16) raw lds[S::RP * S::PITCH];
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
    S now, next;
    if (k0 < k1)
        now.load(c, m, x, j0, k0, kg, on);
    for (int kc = k0; kc < k1; kc += kKC) {
        __syncthreads();  // the chunk before is read
        now.stage(lds);
        if (kc + kKC < k1)
            next.load(c, m, x, j0, kc + kKC, kg, on);
        __syncthreads();
        if (on)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const Raw8<E> mr = *(const Raw8<E> *)(lds + (j * 16 + r15) * S::PITCH + s * 32 + kg * 8);
                    acc[j] = product32<E, X>(mr, now.x[s], acc[j]);
                }
        now = next;
    }
    if (w * 16 + r15 < tl.rows) {
        float *out = c.part + ((int64_t)blockIdx.y * c.o.T + tl.row0 + w * 16 + r15) * c.r + j0;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + j * 16 + kg * 4 + e < c.r)
                    out[j * 16 + kg * 4 + e] = acc[j][e];
    }
}

// ---- expand ----------------------------------------------------------------------------
// grid: tiles times slices of 512 columns, a tile's next to each other.  h of its 64 tokens lies in LDS; a wave has 128
// columns: row m of MFMA e is column 32 (m % 4) + 8 (m / 4) + e, so that the eight MFMAs leave
// a lane four times eight columns in a row, next to those of the lanes of the same token
// (a lane with 32 in a row stores a quarter of each 64 bytes at a time: 4096 tokens of 4096
// columns in bf16 30 against 26 us).  M comes straight from memory into operands (the tiles of an
// adapter share it in the caches) and is held over the tile's tokens up to rank 64.
// SPREAD, for few tiles: slices of 128 columns, the waves share the tokens, 16 each.
//
// A step is 32 places of the reduction.  bf16: the ranks, rounded up to 16 or a multiple of 32
// (rp), follow each other once for each part of h, M is repeated.  Others: 32 ranks in fp32
// products, or 16 where there are no more (HALF: a lane has 4 places instead of 8).
struct ExpandShape {
    int rp, steps, pitch;  // ranks with padding, steps over them (bf16: over all parts), elements per row of h
};
template <bool BF>
__host__ __device__ __forceinline__ ExpandShape expand_shape(int r)
{
    const int rp = r <= 16 ? 16 : (r + 31) / 32 * 32;
    const int steps = BF ? (kParts * rp + 31) / 32 : (rp + 31) / 32;
    return {rp, steps, BF ? steps * 32 + 8 : rp + 4};
}

// M's operands of one step: of eight MFMAs, 8 places of the reduction each
template <class E>
struct Operands {
    Raw8<E> v[8];
};
// Places j .. j + 7 of columns col + e (HALF: j .. j + 3, j a multiple of 4).  OF_A: M lies as [rank][column]; a lane
// reads eight columns of eight ranks and turns them.
template <class E, bool OF_A, bool FULL, bool RFULL, bool HALF>
__device__ __forceinline__ Operands<E> operands(const ExpandCall &c, const typename E::raw *m, int col, int j)
{
    Operands<E> o;
    if constexpr (!OF_A) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o.v[e] = row8<E, RFULL>(m + (int64_t)min(col + e, c.N - 1) * c.r, HALF ? j & ~7 : j, c.r);
            if constexpr (HALF)
                if (j & 4) {
                    if constexpr (sizeof(typename E::raw) == 2)
                        o.v[e].v[0] = u32x4_t{o.v[e].v[0][2], o.v[e].v[0][3], 0, 0};
                    else
                        o.v[e].v[0] = o.v[e].v[1];
                }
        }
    } else {
        constexpr int U = HALF ? 4 : 8;
        Raw8<E> t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = row8<E, FULL>(m + (int64_t)min(j + u, c.r - 1) * c.N, col, c.N);
            if (j + u >= c.r)
                t[u] = Raw8<E>{};
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (sizeof(typename E::raw) == 2) {
#pragma unroll
                for (int q = 0; q < U / 2; ++q)
                    o.v[e].v[0][q] = __builtin_amdgcn_perm(t[2 * q + 1].v[0][e >> 1], t[2 * q].v[0][e >> 1],
                                                           e & 1 ? 0x07060302 : 0x05040100);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    o.v[e].v[u >> 2][u & 3] = t[u].v[e >> 2][e & 3];
            }
        }
    }
    return o;
}

// Three blocks a CU where that costs no spills (146 + 32 registers without, two blocks: 4096 tokens
// 25.9 against 23.3 us).
template <class E, class O, int SETS>
constexpr int kExpandWaves = std::is_same<E, BF16>::value && std::is_same<O, BF16>::value && SETS == 1 ? 3 : 1;

// SETS: steps' worth of M held over the tokens (ranks up to 32 or 64), 0: read again for each 16 tokens
template <class E, class O, bool OF_A, bool FULL, bool RFULL, int SETS, bool HALF, bool SPREAD>
__global__ __launch_bounds__(256, (kExpandWaves<E, O, SETS>)) void k_expand(ExpandCall c)
{
    constexpr bool BF = std::is_same<E, BF16>::value;
    typedef typename std::conditional<BF, uint16_t, float>::type hraw;
    extern __shared__ __align__(16) char smem[];
    hraw *hl = (hraw *)smem;
    const int slices = !c.out ? 1 : SPREAD ? (c.N + 127) / 128 : (c.N + kCols - 1) / kCols;
    const int tile = blockIdx.x / slices, slice = blockIdx.x % slices;
    const Tile tl = tile_of(c.o, tile);
    if (tl.rows <= 0)
        return;
    const ExpandShape sh = expand_shape<BF>(c.r);
    const int tid = threadIdx.x, lane = tid & 63, r15 = lane & 15, kg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool none = tl.a >= c.o.n;  // the tokens without an adapter
    const int a = none ? 0 : tl.a;
    const float scale = none ? 0.f : scale_of(c.scale, a);
    const typename E::raw *m = (const typename E::raw *)c.m + (int64_t)a * c.r * c.N;
    const int c0 = SPREAD ? slice * 128 : slice * kCols + w * 128;
    const bool on = c.out && c0 < c.N;
    // the tokens of this wave's 16s, and their residuals, on their way while h is made
    constexpr int NB = SPREAD ? 1 : 4;
    const int col = c0 + kg * 8, mcol = c0 + 32 * (r15 & 3) + 8 * (r15 >> 2);
    int64_t token[NB];
    Raw8<O> res[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        token[b] = c.o.order[tl.row0 + min((SPREAD ? w : b) * 16 + r15, tl.rows - 1)];
    // a step's place of this lane's first rank
    const auto rank_of = [&](int step) {
        return HALF ? kg * 4 : BF && sh.rp == 16 ? kg * 8 & 8 : (step * 32) % sh.rp + kg * 8;
    };
    Operands<E> held[SETS ? SETS : 1];
    if (on) {
        if (c.residual)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    res[b][i] = row8<O, FULL>((const typename O::raw *)c.residual + token[b] * c.ldres, col + 32 * i, c.N);
        if (SETS > 0 && !none)
#pragma unroll
            for (int q = 0; q < SETS; ++q)
                held[q] = operands<E, OF_A, FULL, RFULL, HALF>(c, m, mcol, rank_of(q));
    }
    // h of the tile's tokens, four ranks at a time: the splits' sum, written out once
    const int quads = sh.rp / 4;
    for (int i = tid; i < kTileRows * quads; i += 256) {
        const int row = i / quads, j = (i - row * quads) * 4;
        f32x4a v = {0.f, 0.f, 0.f, 0.f};
        if (row < tl.rows && j < c.r) {
            if (!none) {
                f32x4a p[kShrinkSplits];
#pragma unroll
                for (int s = 0; s < kShrinkSplits; ++s) {
                    const float *at = c.part + (min(s, c.splits - 1) * (int64_t)c.o.T + tl.row0 + row) * c.r + j;
                    if (c.r % 4 == 0)
                        p[s] = *(const f32x4a *)at;
                    else
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            p[s][q] = at[min(q, c.r - 1 - j)];
                }
#pragma unroll
                for (int s = 0; s < kShrinkSplits; ++s)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] += s < c.splits && j + q < c.r ? p[s][q] : 0.f;
            }
            if (c.h && slice == 0) {
                float *at = c.h + (int64_t)c.o.order[tl.row0 + row] * c.r + j;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (j + q < c.r)
                        at[q] = c.scaled ? v[q] * scale : v[q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] *= scale;
        }
        hraw *at = hl + row * sh.pitch + j;
        if constexpr (BF) {
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float left = v[q];
                    at[p * sh.rp + q] = bf16_part(left);
                    v[q] = left;
                }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                at[q] = v[q];
        }
    }
    if constexpr (BF) {  // the parts end in a whole step
        const int slots = kParts * sh.rp, more = sh.steps * 32 - slots;
        for (int i = tid; i < kTileRows * more; i += 256)
            hl[i / more * sh.pitch + slots + i % more] = 0;
    }
    __syncthreads();
    if (!on)
        return;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int row = (SPREAD ? w : b) * 16 + r15;
        if (row - r15 >= tl.rows)
            break;
        f32x4a acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] = f32x4a{0.f, 0.f, 0.f, 0.f};
        const auto step_of = [&](int s, const Operands<E> &o) __attribute__((always_inline)) {
            if constexpr (BF) {
                const u32x4_t h = *(const u32x4_t *)(hl + row * sh.pitch + s * 32 + kg * 8);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] = mfma_bf16(o.v[e].v[0], h, acc[e]);
            } else {
                constexpr int P = HALF ? 4 : 8;
                float h[P];
#pragma unroll
                for (int i = 0; i < P; ++i)
                    h[i] = hl[row * sh.pitch + s * 32 + kg * P + i];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v[8];
                    widen8<E>(o.v[e], v);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        acc[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[i], h[i], acc[e], 0, 0, 0);
                }
            }
        };
        if (!none) {
            if constexpr (SETS == 0) {
                for (int s = 0; s < sh.steps; ++s)
                    step_of(s, operands<E, OF_A, FULL, RFULL, HALF>(c, m, mcol, rank_of(s)));
            } else {
                // a part's steps, then the next part's over the same operands
                for (int s = 0; s < sh.steps; s += SETS)
#pragma unroll
                    for (int q = 0; q < SETS; ++q)
                        step_of(s + q, held[q]);
            }
        }
        if (row < tl.rows) {
            typename O::raw *out = (typename O::raw *)c.out + token[b] * c.ldout;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (c.residual)
                    widen8<O>(res[b][i], v);
                if (!none)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] += acc[e][i];
                store8<O>(out, col + 32 * i, max(0, min(8, c.N - col - 32 * i)), v);
            }
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

// Both products in one launch where a token's A is small: every block of a token makes h
// itself.  grid: slices of 1024 columns, tokens; sixteen waves share the ranks (fewer ranks: K
// too), then a thread has a column.  What a column needs of B and the residual is on its way
// meanwhile.  Against two kernels see kFewBytes.
template <class E, class O, bool FULL, bool RFULL>
__global__ __launch_bounds__(1024) void k_few(ShrinkCall c, ExpandCall x)
{
    __shared__ float sums[256 + 16], h[256 + 8];
    const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = blockIdx.x * kFewCols + tid, a = adapter_at(c.o, t);
    const bool none = a < 0, in = n < x.N;
    const float scale = none ? 0.f : scale_of(x.scale, a);
    const typename E::raw *up = (const typename E::raw *)x.m + ((int64_t)max(a, 0) * x.N + min(n, x.N - 1)) * c.r;
    Raw8<E> first[2];
    float y = 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        first[q] = row8<E, RFULL>(up, 8 * q, c.r);
    if (x.residual && in)
        y = O::to_f(((const typename O::raw *)x.residual)[t * x.ldres + n]);
    // parts waves a rank
    const int parts = c.r > 8 ? 1 : c.r > 4 ? 2 : c.r > 2 ? 4 : c.r > 1 ? 8 : 16, ranks = 16 / parts;
    if (!none)
        for (int j = w / parts; j < c.r; j += ranks) {
            const typename E::raw *m = (const typename E::raw *)c.m + ((int64_t)a * c.r + j) * c.K;
            const typename E::raw *xr = (const typename E::raw *)c.x + (int64_t)t * c.ldx;
            float s = 0.f;
#pragma unroll 4
            for (int k = (w % parts * 64 + lane) * 8; k < c.K; k += parts * 512) {
                float u[8], v[8];
                const Raw8<E> mr = row8<E, FULL>(m, k, c.K), xv = row8<E, FULL>(xr, k, c.K);
                widen8<E>(mr, u);
                widen8<E>(xv, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s = fmaf(u[i], v[i], s);
            }
            s = wave_sum_f32(s);
            if (lane == 0)
                sums[j * parts + w % parts] = s;
        }
    __syncthreads();
    for (int j = tid; j < (c.r + 7) / 8 * 8; j += 1024) {
        float v = 0.f;
        if (!none && j < c.r)
            for (int q = 0; q < parts; ++q)
                v += sums[j * parts + q];
        h[j] = v;
        if (x.h && blockIdx.x == 0 && j < c.r)
            x.h[(int64_t)t * c.r + j] = v;
    }
    __syncthreads();
    if (!in)
        return;
    if (!none) {
        float s = 0.f;
        for (int j = 0; j < c.r; j += 8) {
            float u[8];
            widen8<E>(j == 0 ? first[0] : j == 8 ? first[1] : row8<E, RFULL>(up, j, c.r), u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(u[i], h[j + i], s);
        }
        y += scale * s;
    }
    ((typename O::raw *)x.out)[t * x.ldout + n] = O::from_f(y);
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
// grid: slices of 128 columns (of one call, then of the other's), runs of the sorted rows
// times `share`, chunks of 64 ranks.  A block takes every share-th adapter of its run; in an
// adapter's part of the run the four waves take 32 tokens in turn and their sums meet in LDS.  An adapter whose tokens all lie in the run is done; the sums of
// one that goes on in other runs are left in the run's slot 0 (it began in an earlier one)
// or 1 and added by k_outer_join.  A lane has column 8 (lane % 16) + e of the slice in MFMA e
// and reads 8 columns of 8 tokens.
struct OuterPair {
    OuterCall c[2];
    int slices;  // of the first
    int per;     // rows per run, of both
    int share;   // blocks that share a run's adapters
};

template <class X, int NJ, bool FULL>
__global__ __launch_bounds__(256) void k_outer(OuterPair two)
{
    constexpr bool BF = std::is_same<X, BF16>::value;
    constexpr int RP = NJ * 16, PITCH = RP + 4;
    __shared__ __align__(16) float sums[2][kOuterCols * PITCH];  // [column][rank]
    const bool second = (int)blockIdx.x >= two.slices;
    const OuterCall &c = two.c[second];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r15 = lane & 15, kg = lane >> 4;
    const int c0 = (blockIdx.x - (second ? two.slices : 0)) * kOuterCols, j0 = blockIdx.z * kRC;
    const int run = blockIdx.y / two.share, turn = blockIdx.y % two.share;
    const int beg = run * two.per, stop = beg + two.per;  // (an adapter's rows end by themselves)
    const auto adapter = [&](int a, int o0, int o1) __attribute__((always_inline)) {
        const int s0 = max(o0, beg), s1 = min(o1, stop);
        f32x4a acc[NJ][8];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[j][e] = f32x4a{0.f, 0.f, 0.f, 0.f};
        const float gs = scale_of(c.gscale, a);
        // (x of the next 32 tokens is under way over the products of these)
        int t[8];
        Raw8<X> next[8];
        const auto tokens = [&](int t0) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                t[u] = c.o.order[min(t0 + 8 * kg + u, s1 - 1)];
        };
        const auto read = [&]() {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                next[u] = row8<X, FULL>((const typename X::raw *)c.x + t[u] * c.ldx, c0 + 8 * r15, c.W);
        };
        const int first = s0 + w * 32;
        if (first < s1) {
            tokens(first);
            read();
        }
        for (int t0 = first; t0 < s1; t0 += 4 * 32) {
            Raw8<X> xr[8];
            float g[NJ][8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const bool in = t0 + 8 * kg + u < s1;
                xr[u] = next[u];
                if (!in)
                    xr[u] = Raw8<X>{};
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int at = j0 + j * 16 + r15;
                    const float v = c.g[(int64_t)t[u] * c.r + min(at, c.r - 1)];
                    g[j][u] = at < c.r && in ? v * gs : 0.f;
                }
            }
            if (t0 + 4 * 32 < s1) {
                tokens(t0 + 4 * 32);
                read();
            }
            if constexpr (BF) {
                u32x4_t gp[NJ][kParts];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
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
                        for (int p = 0; p < kParts; ++p)
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
        // the sums of waves 0 and 1, then those of 2 and 3 onto them
        for (int q = 0; q < 2; ++q) {
            if (w >> 1 == q)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f32x4a *at = (f32x4a *)(sums[w & 1] + (8 * r15 + e) * PITCH + j * 16 + kg * 4);
                        if (q) {
                            const f32x4a v = *at;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[j][e][i] += v[i];
                        }
                        *at = acc[j][e];
                    }
            __syncthreads();
        }
        const bool whole = o0 >= beg && o1 <= stop;
        float *slot = c.slots + ((int64_t)run * 2 + (o0 >= beg)) * c.r * c.W;
        for (int i = tid; i < RP * kOuterCols; i += 256) {
            // along the side that is contiguous
            const int j = c.of_b ? i % RP : i / kOuterCols, x = c.of_b ? i / RP : i % kOuterCols;
            if (j0 + j >= c.r || c0 + x >= c.W)
                continue;
            const float v = sums[0][x * PITCH + j] + sums[1][x * PITCH + j];
            const int64_t at = c.of_b ? (int64_t)(c0 + x) * c.r + j0 + j : (int64_t)(j0 + j) * c.W + c0 + x;
            if (whole)
                store_el(c.d, (int64_t)a * c.r * c.W + at, v, c.grad_dtype);
            else
                slot[at] = v;
        }
        __syncthreads();
    };
    // this block's adapters with rows in the run, found 64 at a time
    for (int e0 = 0; e0 < c.o.n; e0 += 64) {
        const int e = e0 + lane, from = c.o.offsets[min(e, c.o.n)], to = c.o.offsets[min(e + 1, c.o.n)];
        uint64_t mine = __ballot(e < c.o.n && e % two.share == turn && max(from, beg) < min(to, stop));
        for (; mine; mine &= mine - 1) {
            const int i = __ffsll((unsigned long long)mine) - 1;
            adapter(e0 + i, __builtin_amdgcn_readlane(from, i), __builtin_amdgcn_readlane(to, i));
        }
    }
}

// grid: blocks of 256 elements (of one call, then of the other's), adapters
__global__ __launch_bounds__(256) void k_outer_join(OuterPair two)
{
    const int64_t blocks = ((int64_t)two.c[0].r * two.c[0].W + 255) / 256;
    const bool second = blockIdx.x >= blocks;
    const OuterCall &c = two.c[second];
    const int a = blockIdx.y;
    const int o0 = c.o.offsets[a], o1 = c.o.offsets[a + 1];
    const int first = o0 / two.per, last = (o1 - 1) / two.per;
    if (o1 > o0 && first == last)
        return;
    const int64_t size = (int64_t)c.r * c.W, i = (blockIdx.x - (second ? blocks : 0)) * 256 + threadIdx.x;
    if (i >= size)
        return;
    float v = 0.f;
    if (o1 > o0)
#pragma unroll 16
        for (int q = first; q <= last; ++q)
            v += c.slots[((int64_t)q * 2 + (q == first)) * size + i];
    store_el(c.d, (int64_t)a * size + i, v, c.grad_dtype);
}

// ---- launches --------------------------------------------------------------------------

int most_tiles(const AdapterOrder &o) { return o.T / kTileRows + (o.n + 1 < o.T ? o.n + 1 : o.T); }
int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

// (RFULL: whether rows of M of r elements, which only the transpose has, are whole chunks)
template <class E, class X, bool OF_B, bool FULL, bool RFULL>
void shrink_of(const ShrinkCall &c, hipStream_t st)
{
    const dim3 grid(most_tiles(c.o), c.splits, (c.r + kRC - 1) / kRC);
    switch (rank_blocks(c.r)) {
    case 1: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 1, FULL, RFULL>), grid, dim3(256), 0, st, c); break;
    case 2: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 2, FULL, RFULL>), grid, dim3(256), 0, st, c); break;
    default: hipLaunchKernelGGL((k_shrink<E, X, OF_B, 4, FULL, RFULL>), grid, dim3(256), 0, st, c);
    }
}

template <class E, class O, bool OF_A, bool FULL, bool RFULL>
void expand_of(const ExpandCall &c, hipStream_t st)
{
    constexpr bool BF = std::is_same<E, BF16>::value;
    // fewer than a block a CU: the columns in four times as many slices
    const int tiles = most_tiles(c.o), slices = (c.N + kCols - 1) / kCols;
    const bool spread = c.out && c.r <= 64 && (c.o.T / kTileRows + 1) * slices < 256;
    const dim3 grid(tiles * (!c.out ? 1 : spread ? (c.N + 127) / 128 : slices));
    const size_t lds = (size_t)kTileRows * expand_shape<BF>(c.r).pitch * (BF ? 2 : 4);
    with_bool(spread, [&](auto sp) {
        constexpr bool SP = decltype(sp)::value;
        if (c.r <= 16)
            hipLaunchKernelGGL((k_expand<E, O, OF_A, FULL, RFULL, 1, !BF, SP>), grid, dim3(256), lds, st, c);
        else if (c.r <= 32)
            hipLaunchKernelGGL((k_expand<E, O, OF_A, FULL, RFULL, 1, false, SP>), grid, dim3(256), lds, st, c);
        else if (c.r <= 64)
            hipLaunchKernelGGL((k_expand<E, O, OF_A, FULL, RFULL, 2, false, SP>), grid, dim3(256), lds, st, c);
        else if constexpr (!SP)
            hipLaunchKernelGGL((k_expand<E, O, OF_A, FULL, RFULL, 0, false, false>), grid, dim3(256), lds, st, c);
    });
}

template <class X, bool FULL>
void outer_of(const OuterPair &p, int slices, int chunks, hipStream_t st)
{
    const int r = p.c[0].r;
    const dim3 grid(slices, chunks * p.share, (r + kRC - 1) / kRC);
    switch (rank_blocks(r)) {
    case 1: hipLaunchKernelGGL((k_outer<X, 1, FULL>), grid, dim3(256), 0, st, p); break;
    case 2: hipLaunchKernelGGL((k_outer<X, 2, FULL>), grid, dim3(256), 0, st, p); break;
    default: hipLaunchKernelGGL((k_outer<X, 4, FULL>), grid, dim3(256), 0, st, p);
    }
}

}  // namespace

int launch_shrink(const ShrinkCall &c, hipStream_t st)
{
    ProfScope prof("adapter_shrink", st);
    with_bool(c.K % 8 == 0, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (c.of_b)
            with_bool(c.r % 8 == 0, [&](auto rfull) {
                constexpr bool RFULL = decltype(rfull)::value;
                with_pair(c.dtype, c.x_dtype, [&](auto e, auto x) { shrink_of<decltype(e), decltype(x), true, FULL, RFULL>(c, st); });
            });
        else
            with_element(c.dtype, [&](auto e) { shrink_of<decltype(e), decltype(e), false, FULL, true>(c, st); });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_expand(const ExpandCall &c, hipStream_t st)
{
    ProfScope prof("adapter_expand", st);
    with_bool(c.N % 8 == 0, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (c.of_a)
            with_element(c.dtype, [&](auto e) { expand_of<decltype(e), decltype(e), true, FULL, true>(c, st); });
        else
            with_bool(c.r % 8 == 0, [&](auto rfull) {
                constexpr bool RFULL = decltype(rfull)::value;
                with_pair(c.dtype, c.out_dtype, [&](auto e, auto o) { expand_of<decltype(e), decltype(o), false, FULL, RFULL>(c, st); });
            });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_few(const ShrinkCall &c, const ExpandCall &x, hipStream_t st)
{
    ProfScope prof("adapter_few", st);
    const dim3 grid((x.N + kFewCols - 1) / kFewCols, c.o.T);
    with_bool(c.K % 8 == 0, [&](auto full) {
        with_bool(c.r % 8 == 0, [&](auto rfull) {
            with_pair(x.dtype, x.out_dtype, [&](auto e, auto o) {
                hipLaunchKernelGGL((k_few<decltype(e), decltype(o), decltype(full)::value, decltype(rfull)::value>), grid, dim3(1024),
                                   0, st, c, x);
            });
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

int launch_outer(const OuterCall *calls, int n, int chunks, hipStream_t st)
{
    ProfScope prof("adapter_outer", st);
    OuterPair p{};
    p.c[0] = calls[0], p.c[1] = calls[n - 1];
    p.slices = outer_slices(calls[0].W);
    const int T = calls[0].o.T;
    p.per = T > 0 ? ((T + chunks - 1) / chunks + 31) / 32 * 32 : 32;
    int slices = 0;
    int64_t blocks = 0;
    bool whole = true;
    for (int i = 0; i < n; ++i) {
        slices += outer_slices(calls[i].W);
        blocks += ((int64_t)calls[i].r * calls[i].W + 255) / 256;
        whole = whole && calls[i].W % 8 == 0;
    }
    // Many adapters in a run are shared by blocks: by as many as fill the GPU, and so that one has about
    // four to do (39 tokens of 15 adapters, 219 to 768 in fp16 at rank 64: 285 us by one block a run, 40 so).
    const int n_adapters = calls[0].o.n, room = 512 / (slices * chunks), each = n_adapters / (4 * chunks);
    p.share = each > 16 ? 16 : each;
    p.share = p.share > room ? p.share : room;
    p.share = p.share < n_adapters ? p.share : n_adapters;
    p.share = p.share > 1 ? p.share : 1;
    with_bool(whole, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        if (calls[0].x_dtype == ECF_BF16)
            outer_of<BF16, FULL>(p, slices, chunks, st);
        else if (calls[0].x_dtype == ECF_F32)
            outer_of<F32, FULL>(p, slices, chunks, st);
        else
            outer_of<F16, FULL>(p, slices, chunks, st);
    });
    ECF_HIP_CHECK(hipGetLastError());
    hipLaunchKernelGGL(k_outer_join, dim3((unsigned)blocks, calls[0].o.n), dim3(256), 0, st, p);
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

}  // namespace ecf
