// Tokens to experts and back: the stable sort of their choices, dispatch, combine and its
// gradient.
//
// The sort is a counting sort.  A wave ranks 64 choices at a time: lanes with the same
// expert find each other by a ballot per bit of its number, and a choice's place is the
// expert's first row + the rows of it in earlier segments, waves and steps + its rank among
// its peers, so equal choices keep their order.  A choice of no expert has number E.
//
// Dispatch reads each token once and writes its k rows; combine reads a token's k rows
// with all loads under way together and adds them in ascending j.
#include "tokens_device.h"

namespace ecf {
namespace {

constexpr int kSortOne = 4096;      // choices up to which one block sorts them all
constexpr int kSortSegments = 128;  // most segments
constexpr int kSortRows = 1024;     // choices that a block takes at a time

__device__ __forceinline__ int choice(const SortCall &c, int64_t f)
{
    const int64_t t = f / c.k, at = t * c.ldidx + (f - t * c.k);
    const int64_t e = c.wide ? ((const int64_t *)c.idx)[at] : ((const int32_t *)c.idx)[at];
    return e >= 0 && e < c.E ? (int)e : c.E;
}

__device__ __forceinline__ uint64_t peers_of(int key, bool valid, int bits)
{
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool bit = (key >> b) & 1;
        const uint64_t v = __ballot(valid && bit);
        m &= bit ? v : ~v;
    }
    return valid ? m : 0ull;
}

// Exclusive sums over the block's 1024 threads of two counts at once (each below 2^31 in
// total); sh: 17 values.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *sh, uint64_t *total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up(x, o, 64);
        x += lane >= o ? y : 0;
    }
    if (lane == 63)
        sh[w] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint64_t s = sh[i];
        before += i < w ? s : 0;
        all += s;
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

__global__ __launch_bounds__(1024) void k_token_count(SortCall c, int64_t per)
{
    extern __shared__ int hist[];  // [E + 1]
    for (int e = threadIdx.x; e <= c.E; e += 1024)
        hist[e] = 0;
    __syncthreads();
    const int64_t rows = (int64_t)c.T * c.k, end = min(rows, ((int64_t)blockIdx.x + 1) * per);
    for (int64_t f = (int64_t)blockIdx.x * per + threadIdx.x; f < end; f += 1024)
        atomicAdd(&hist[choice(c, f)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= c.E; e += 1024)
        c.segments[(int64_t)blockIdx.x * (c.E + 1) + e] = hist[e];
}

// Each block places its segment; block 0 writes the tables.  segments: the counts of all
// segments (one segment: counted here).  A wave owns a run of its segment's choices.
__global__ __launch_bounds__(1024) void k_token_place(SortCall c, int64_t per, int segments, int bits)
{
    extern __shared__ int base[];  // [16][E + 1]
    __shared__ uint64_t sh[17];
    const int EB = c.E + 1, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t rows = (int64_t)c.T * c.k, beg = (int64_t)blockIdx.x * per, end = min(rows, beg + per);
    const int64_t run = ((per + 15) / 16 + 63) / 64 * 64, wb = min(end, beg + w * run), we = min(end, wb + run);
    for (int i = tid; i < 16 * EB; i += 1024)
        base[i] = 0;
    __syncthreads();
    for (int64_t f = wb + lane; f < we; f += 64)
        atomicAdd(&base[w * EB + choice(c, f)], 1);
    __syncthreads();
    // expert tid's rows, those before this segment, and its first row
    int all = 0, before = 0;
    if (tid < c.E) {
        if (segments == 1)
            for (int q = 0; q < 16; ++q)
                all += base[q * EB + tid];
        else
#pragma unroll 8
            for (int s = 0; s < segments; ++s) {
                const int v = c.segments[(int64_t)s * EB + tid];
                all += v;
                before += s < (int)blockIdx.x ? v : 0;
            }
    }
    uint64_t total;
    const uint64_t first = block_scan((uint64_t)all | (uint64_t)((all + kTileRows - 1) / kTileRows) << 32, sh, &total);
    const int chosen = (int)(uint32_t)total;
    if (blockIdx.x == 0) {
        if (tid < c.E) {
            c.counts[tid] = all;
            c.offsets[tid] = (int)(uint32_t)first;
            c.tiles[tid] = (int)(first >> 32);
        }
        if (tid == 0) {
            const int none = (int)(rows - chosen), tiles = (int)(total >> 32);
            c.offsets[c.E] = chosen;
            c.tiles[c.E] = tiles;
            c.tiles[c.E + 1] = tiles + (none + kTileRows - 1) / kTileRows;
        }
    }
    // the first row of each wave's choices of each expert
    if (tid < c.E) {
        int at = (int)(uint32_t)first + before;
        for (int q = 0; q < 16; ++q) {
            const int v = base[q * EB + tid];
            base[q * EB + tid] = at;
            at += v;
        }
    }
    // (those of no expert by the last thread, which may have an expert as well)
    if (tid == 1023) {
        int at = chosen;
        if (segments > 1)
            for (int s = 0; s < (int)blockIdx.x; ++s)
                at += c.segments[(int64_t)s * EB + c.E];
        for (int q = 0; q < 16; ++q) {
            const int v = base[q * EB + c.E];
            base[q * EB + c.E] = at;
            at += v;
        }
    }
    __syncthreads();
    for (int64_t f0 = wb; f0 < we; f0 += 64) {
        const int64_t f = f0 + lane;
        const bool valid = f < we;
        const int key = valid ? choice(c, f) : 0;
        const uint64_t peers = peers_of(key, valid, bits);
        if (valid) {
            const int b = base[w * EB + key], p = b + __popcll(peers & lanemask_lt(lane));
            c.order[p] = (int)f;
            c.place[f] = p;
            if (lane == __ffsll((unsigned long long)peers) - 1)
                base[w * EB + key] = b + __popcll(peers);
        }
    }
}

// ---- dispatch --------------------------------------------------------------------------

// Eight elements of an e4m3 row from column col on (zeros past its end), times their scale.
template <bool FULL>
__device__ __forceinline__ void mx8(const uint8_t *row, const uint8_t *scale, int64_t col, int d, float v[8])
{
    uint32_t p[2] = {0, 0};
    if (FULL || col + 8 <= d) {
        struct __attribute__((packed, aligned(1))) any64 {
            uint32_t v[2];
        };
        const any64 a = *(const any64 *)(row + col);
        p[0] = a.v[0], p[1] = a.v[1];
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col + j < d)
                p[j >> 2] |= (uint32_t)row[col + j] << (8 * (j & 3));
    }
    const float s = mx_scale(scale[col / 32]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[h], true);
        v[4 * h] = a[0] * s, v[4 * h + 1] = a[1] * s, v[4 * h + 2] = b[0] * s, v[4 * h + 3] = b[1] * s;
    }
}

// grid: 2^shift threads per token, 256 in a block
template <class E, bool MX, bool FULL>
__global__ __launch_bounds__(256) void k_dispatch(MoveCall c, int shift)
{
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= c.T)
        return;
    const int G = 1 << shift;
    const int n_rows = *c.n_rows;
    const int64_t all = (int64_t)c.T * c.k;
    for (int64_t col = (threadIdx.x & (G - 1)) * 8; col < c.d; col += G * 8) {
        float v[8];
        if constexpr (MX)
            mx8<FULL>((const uint8_t *)c.x + t * c.ldx, (const uint8_t *)c.x_scale + t * c.ldxs, col, c.d, v);
        else
            widen8<E>(row8<E, FULL>((const typename E::raw *)c.x + t * c.ldx, col, c.d), v);
        const int n = (int)min((int64_t)8, c.d - col);
        for (int j0 = 0; j0 < c.k; j0 += 8) {
            int p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                p[u] = c.place[t * c.k + min(j0 + u, c.k - 1)];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j0 + u < c.k && (uint32_t)p[u] < (uint64_t)all) {
                    const bool none = p[u] >= n_rows;
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = none ? 0.f : v[i];
                    store8<E>((typename E::raw *)c.rows + p[u] * c.ldrows, col, n, y);
                }
        }
    }
}

// ---- combine ---------------------------------------------------------------------------

template <class E, class O, bool FULL>
__global__ __launch_bounds__(256) void k_combine_tokens(MoveCall c, int shift)
{
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= c.T)
        return;
    const int G = 1 << shift;
    const int n_rows = *c.n_rows;
    for (int64_t col = (threadIdx.x & (G - 1)) * 8; col < c.d; col += G * 8) {
        const int n = (int)min((int64_t)8, c.d - col);
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c.residual)
            widen8<O>(row8<O, FULL>((const typename O::raw *)c.residual + t * c.ldres, col, c.d), r);
        for (int j0 = 0; j0 < c.k; j0 += 8) {
            Raw8<E> y[8];
            bool use[8];
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t f = t * c.k + min(j0 + u, c.k - 1);
                const int p = c.place[f];
                use[u] = j0 + u < c.k && (uint32_t)p < (uint32_t)n_rows;
                w[u] = c.weight ? c.weight[f] : 1.f;
                // a choice of no expert: the first row, left out below (there is one: n_rows may be 0, T k is not)
                y[u] = row8<E, FULL>((const typename E::raw *)c.rows + (use[u] ? p : 0) * c.ldrows, col, c.d);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float v[8];
                widen8<E>(y[u], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i] = use[u] ? fmaf(w[u], v[i], s[i]) : s[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = r[i] + s[i];
        store8<O>((typename O::raw *)c.out + t * c.ldout, col, n, s);
    }
}

// grid: one wave per choice
template <class E, class O, bool FULL>
__global__ __launch_bounds__(256) void k_combine_back(MoveCall c)
{
    const int64_t f = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), all = (int64_t)c.T * c.k;
    if (f >= all)
        return;
    const int lane = threadIdx.x & 63;
    const int64_t t = f / c.k;
    const int p = c.place[f];
    const bool none = p >= *c.n_rows, there = (uint32_t)p < (uint64_t)all;
    const float w = c.weight ? c.weight[f] : 1.f;
    const typename O::raw *dout = (const typename O::raw *)c.dout + t * c.lddout;
    const typename E::raw *y = (const typename E::raw *)c.rows + (there ? p : 0) * c.ldrows;
    typename E::raw *dr = (typename E::raw *)c.drows + (there ? p : 0) * c.lddrows;
    const bool dots = c.dweight && !none && there;
    double dot = 0.0;
    for (int64_t c0 = 0; c0 < c.d; c0 += 64 * 8) {
        const int64_t col = c0 + lane * 8;
        float g[8], v[8];
        const Raw8<O> gr = row8<O, FULL>(dout, col, c.d);
        if (dots) {
            const Raw8<E> yr = row8<E, FULL>(y, col, c.d);
            widen8<O>(gr, g);
            widen8<E>(yr, v);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(g[i], v[i], s);
            dot += (double)s;
        } else {
            widen8<O>(gr, g);
        }
        if (c.drows && there) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = none ? 0.f : w * g[i];
            store8<E>(dr, col, (int)max((int64_t)0, min((int64_t)8, c.d - col)), g);
        }
    }
    if (c.dweight) {
        dot = wave_sum_f64(dot);
        if (lane == 0)
            c.dweight[f] = dots ? (float)dot : 0.f;
    }
}

// Threads per token, as a power of two from 8 to 256: a chunk of eight elements each.
int token_shift(int d)
{
    int s = 3;
    while (s < 8 && (8 << s) < d)
        ++s;
    return s;
}

dim3 token_grid(int T, int shift)
{
    const int per = 256 >> shift;
    return dim3((unsigned)((T + per - 1) / per));
}

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
void with_pair(const MoveCall &c, F f)
{
    with_element(c.dtype, [&](auto e) {
        if (c.token_dtype == ECF_F32)
            f(e, F32{});
        else
            f(e, e);
    });
}

}  // namespace

int sort_segments(int64_t rows)
{
    if (rows <= kSortOne)
        return 1;
    const int64_t n = (rows + kSortRows - 1) / kSortRows;
    return (int)(n < kSortSegments ? n : kSortSegments);
}

int launch_token_sort(const SortCall &c, hipStream_t st)
{
    ProfScope prof("token_sort", st);
    const int64_t rows = (int64_t)c.T * c.k;
    const int n = sort_segments(rows);
    const int64_t per = n == 1 ? (rows < kSortRows ? kSortRows : rows) : ((rows + n - 1) / n + kSortRows - 1) / kSortRows * kSortRows;
    const size_t sh = (size_t)(c.E + 1) * 4;
    int bits = 0;
    while ((1 << bits) <= c.E)
        ++bits;
    if (n > 1)
        hipLaunchKernelGGL(k_token_count, dim3(n), dim3(1024), sh, st, c, per);
    hipLaunchKernelGGL(k_token_place, dim3(n), dim3(1024), 16 * sh, st, c, per, n, bits);
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_dispatch(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_dispatch", st);
    const int shift = token_shift(c.d);
    const bool full = c.d % 8 == 0;
    with_element(c.dtype, [&](auto e) {
        using E = decltype(e);
        if (c.token_dtype == ECF_MXFP8) {
            if (full)
                hipLaunchKernelGGL((k_dispatch<E, true, true>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
            else
                hipLaunchKernelGGL((k_dispatch<E, true, false>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
        } else {
            if (full)
                hipLaunchKernelGGL((k_dispatch<E, false, true>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
            else
                hipLaunchKernelGGL((k_dispatch<E, false, false>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
        }
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_combine_tokens(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_combine", st);
    const int shift = token_shift(c.d);
    with_pair(c, [&](auto e, auto o) {
        using E = decltype(e);
        using O = decltype(o);
        if (c.d % 8 == 0)
            hipLaunchKernelGGL((k_combine_tokens<E, O, true>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
        else
            hipLaunchKernelGGL((k_combine_tokens<E, O, false>), token_grid(c.T, shift), dim3(256), 0, st, c, shift);
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_combine_backward(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_combine_backward", st);
    const dim3 grid((unsigned)(((int64_t)c.T * c.k + 3) / 4));
    with_pair(c, [&](auto e, auto o) {
        using E = decltype(e);
        using O = decltype(o);
        if (c.d % 8 == 0)
            hipLaunchKernelGGL((k_combine_back<E, O, true>), grid, dim3(256), 0, st, c);
        else
            hipLaunchKernelGGL((k_combine_back<E, O, false>), grid, dim3(256), 0, st, c);
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

}  // namespace ecf
