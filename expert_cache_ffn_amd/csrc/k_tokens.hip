// Tokens to experts and back: the stable sort of their choices, dispatch, combine and its
// gradient.
//
// The sort is a counting sort.  A wave ranks 64 choices at a time: lanes with the same
// expert find each other by a ballot per bit of its number, and a choice's place is the
// expert's first row + the rows of it in earlier segments, waves and steps + its rank among
// its peers, so equal choices keep their order.  A choice of no expert has number E.
//
// Dispatch reads each token once and writes its k rows (a gather by rows would read it k
// times); combine reads a token's k rows with all loads under way together and adds them in
// ascending j; its gradient has a wave per choice, so that a weight's gradient is a sum
// within the wave and the token's dout comes from the caches for its other choices.
//
// Bound by memory: 4096 tokens of 4096 in bf16, top-6, dispatch 43 us (5.5 TB/s), combine onto
// an fp32 sum 70 (4.8); 8192 tokens, top-8, combine's gradient 230 (4.9), dispatch's 113 (5.3);
// a large copy takes 5.0 TB/s.  Sort of 24576 choices of 256 experts 4.9 + 9.3 us, of 96 2.9: the
// latency of its dependent steps.
#include "tokens_device.h"

namespace ecf {
namespace {


__device__ __forceinline__ int choice(const SortCall &c, uint32_t f)
{
    int64_t at = f;
    if (c.ldidx != c.k) {
        const uint32_t t = f / (uint32_t)c.k;
        at = t * c.ldidx + (f - t * (uint32_t)c.k);
    }
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

// What lanes of this wave have written to LDS before is there for all of them after it.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Exclusive sums over the block's threads (NW waves) of two counts at once, each below 2^31 in
// total.
template <int NW>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *sh, uint64_t *total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint64_t x = wave_incl_scan64(v);
    if (lane == 63)
        sh[w] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint64_t s = sh[i];
        before += i < w ? s : 0;
        all += s;
    }
    *total = all;
    return before + x - v;
}

__global__ __launch_bounds__(1024) void k_token_count(SortCall c, uint32_t per)
{
    extern __shared__ int hist[];  // [E + 1]
    for (int e = threadIdx.x; e <= c.E; e += 1024)
        hist[e] = 0;
    __syncthreads();
    const uint32_t rows = (uint32_t)c.T * c.k, beg = blockIdx.x * per, end = min(rows, beg + per);
    for (uint32_t f = beg + threadIdx.x; f < end; f += 1024)
        atomicAdd(&hist[choice(c, f)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= c.E; e += 1024)
        c.segments[(int64_t)blockIdx.x * (c.E + 1) + e] = hist[e];
}

// Each block places its segment; block 0 writes the tables.  A wave owns a run of its
// segment's choices: one step of 64 (HELD), whose numbers and ranks stay in registers, or
// more, which are counted first and ranked in a second pass.  The block has at least E threads.
// SELF: the other segments' choices are counted here; otherwise k_token_count has left the
// counts of each segment.
template <int NW, bool HELD, bool SELF>
__global__ __launch_bounds__(64 * NW) void k_token_place(SortCall c, uint32_t per, int segments, int bits)
{
    extern __shared__ int base[];  // [NW][E + 1], SELF: and the counts of the segments after and before this one
    __shared__ uint64_t sh[NW];
    constexpr int NT = 64 * NW;
    const int EB = c.E + 1, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    int *later = base + NW * EB, *earlier = later + EB;
    const uint32_t rows = (uint32_t)c.T * c.k, beg = min(rows, blockIdx.x * per), end = min(rows, beg + per);
    const uint32_t run = ((per + NW - 1) / NW + 63) / 64 * 64, wb = min(end, beg + w * run), we = min(end, wb + run);
    int key = -1, rank = 0;
    if (HELD && wb + lane < we)
        key = choice(c, wb + lane);
    for (int i = tid; i < (SELF ? NW + 2 : NW) * EB; i += NT)
        base[i] = 0;
    // this expert's rows in the other segments and in those before (loads under way over the barrier)
    int all = 0, before = 0, none_before = 0;
    if constexpr (!SELF) {
        const int col = min(tid, c.E);
#pragma unroll 16
        for (int s = 0; s < segments; ++s) {
            const int v = c.segments[(int64_t)s * EB + col];
            all += s == (int)blockIdx.x ? 0 : v;
            before += s < (int)blockIdx.x ? v : 0;
        }
        // those of no expert, by the last thread, which may have an expert as well
        if (tid == NT - 1)
#pragma unroll 16
            for (int s = 0; s < (int)blockIdx.x; ++s)
                none_before += c.segments[(int64_t)s * EB + c.E];
    }
    __syncthreads();
    if constexpr (SELF) {
        if (segments > 1) {
            for (int s0 = 0; s0 < segments; s0 += 8) {
                int k[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t f = (s0 + q) * per + tid;
                    k[q] = s0 + q != (int)blockIdx.x && s0 + q < segments && f < rows ? choice(c, f) : -1;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (k[q] >= 0)
                        atomicAdd(s0 + q < (int)blockIdx.x ? &earlier[k[q]] : &later[k[q]], 1);
            }
            __syncthreads();
        }
        if (tid <= c.E) {
            before = earlier[tid];
            all = before + later[tid];
        }
        if (tid == NT - 1)
            none_before = earlier[c.E];
    }
    if constexpr (HELD) {
        const uint64_t peers = peers_of(key, key >= 0, bits);
        if (key >= 0) {
            rank = __popcll(peers & lanemask_lt(lane));
            if (rank == 0)
                base[w * EB + key] = __popcll(peers);
        }
    } else {
        for (uint32_t f = wb + lane; f < we; f += 64)
            atomicAdd(&base[w * EB + choice(c, f)], 1);
    }
    __syncthreads();
    // the waves' counts of each expert become what comes before them
    int mine = 0;
    if (tid < c.E)
        for (int q = 0; q < NW; ++q) {
            const int v = base[q * EB + tid];
            base[q * EB + tid] = mine;
            mine += v;
        }
    all = tid < c.E ? all + mine : 0;
    uint64_t total;
    const uint64_t first = block_scan<NW>((uint64_t)all | (uint64_t)((all + kTileRows - 1) / kTileRows) << 32, sh, &total);
    const int chosen = (int)(uint32_t)total;
    if (blockIdx.x == 0) {
        if (tid < c.E) {
            c.counts[tid] = all;
            c.offsets[tid] = (int)(uint32_t)first;
            c.tiles[tid] = (int)(first >> 32);
        }
        if (tid == 0) {
            const int none = (int)rows - chosen, tiles = (int)(total >> 32);
            c.offsets[c.E] = chosen;
            c.tiles[c.E] = tiles;
            c.tiles[c.E + 1] = tiles + (none + kTileRows - 1) / kTileRows;
        }
    }
    if (tid < c.E) {
        const int at = (int)(uint32_t)first + before;
#pragma unroll
        for (int q = 0; q < NW; ++q)
            base[q * EB + tid] += at;
    }
    if (tid == NT - 1) {
        int at = chosen + none_before;
        for (int q = 0; q < NW; ++q) {
            const int v = base[q * EB + c.E];
            base[q * EB + c.E] = at;
            at += v;
        }
    }
    __syncthreads();
    if constexpr (HELD) {
        if (key >= 0) {
            const int p = base[w * EB + key] + rank;
            c.order[p] = (int)(wb + lane);
            c.place[wb + lane] = p;
        }
    } else {
        for (uint32_t f0 = wb; f0 < we; f0 += 64) {
            const uint32_t f = f0 + lane;
            const bool valid = f < we;
            const int e = valid ? choice(c, f) : 0;
            const uint64_t peers = peers_of(e, valid, bits);
            const int b = base[w * EB + e], p = b + __popcll(peers & lanemask_lt(lane));
            if (valid) {
                c.order[p] = (int)f;
                c.place[f] = p;
            }
            wave_sync();  // all lanes have read what one of them now moves on for the next 64
            if (valid && lane == __ffsll((unsigned long long)peers) - 1)
                base[w * EB + e] = b + __popcll(peers);
            wave_sync();
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

// A block has 256 threads, 2^SHIFT of them per token (8: one token), a thread eight columns;
// grid: tokens, groups of columns.
template <int SHIFT>
__device__ __forceinline__ int64_t token_at()
{
    return SHIFT == 8 ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x << (8 - SHIFT)) + (threadIdx.x >> SHIFT);
}
template <int SHIFT>
__device__ __forceinline__ int64_t column_at()
{
    return (((int64_t)blockIdx.y << SHIFT) + (threadIdx.x & ((1 << SHIFT) - 1))) * 8;
}

template <class E, bool MX, bool FULL, int SHIFT>
__global__ __launch_bounds__(256) void k_dispatch(MoveCall c)
{
    const int64_t t = token_at<SHIFT>(), col = column_at<SHIFT>();
    if (t >= c.T || col >= c.d)
        return;
    const int n_rows = *c.n_rows;
    const uint32_t all = (uint32_t)c.T * c.k;
    const int n = (int)min((int64_t)8, c.d - col);
    float v[8];
    if constexpr (MX)
        mx8<FULL>((const uint8_t *)c.x + t * c.ldx, (const uint8_t *)c.x_scale + t * c.ldxs, col, c.d, v);
    else
        widen8<E>(row8<E, FULL>((const typename E::raw *)c.x + t * c.ldx, col, c.d), v);
    for (int j0 = 0; j0 < c.k; j0 += 8) {
        int p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            p[u] = c.place[t * c.k + min(j0 + u, c.k - 1)];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j0 + u < c.k && (uint32_t)p[u] < all) {
                const bool none = p[u] >= n_rows;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = none ? 0.f : v[i];
                store8<E>((typename E::raw *)c.rows + p[u] * c.ldrows, col, n, y);
            }
    }
}

// ---- combine ---------------------------------------------------------------------------

// KN: rows whose loads are under way together, k itself up to 8.
template <class E, class O, bool FULL, int SHIFT, int KN>
__global__ __launch_bounds__(256) void k_combine_tokens(MoveCall c)
{
    const int64_t t = token_at<SHIFT>(), col = column_at<SHIFT>();
    if (t >= c.T || col >= c.d)
        return;
    const int n_rows = *c.n_rows;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c.residual)
        widen8<O>(row8<O, FULL>((const typename O::raw *)c.residual + t * c.ldres, col, c.d), r);
    for (int j0 = 0; j0 < c.k; j0 += KN) {
        Raw8<E> y[KN];
        bool use[KN];
        float w[KN];
#pragma unroll
        for (int u = 0; u < KN; ++u) {
            const int64_t f = t * c.k + min(j0 + u, c.k - 1);
            const int p = c.place[f];
            use[u] = j0 + u < c.k && (uint32_t)p < (uint32_t)n_rows;
            w[u] = c.weight ? c.weight[f] : 1.f;
            // a choice of no expert: the first row, left out below (there is one: n_rows may be 0, T k is not)
            y[u] = row8<E, FULL, true>((const typename E::raw *)c.rows + (use[u] ? p : 0) * c.ldrows, col, c.d);
        }
#pragma unroll
        for (int u = 0; u < KN; ++u) {
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
    store8<O>((typename O::raw *)c.out + t * c.ldout, col, (int)min((int64_t)8, c.d - col), s);
}

// G lanes per choice, 256 threads in a block.
template <class E, class O, bool FULL, int G>
__global__ __launch_bounds__(256) void k_combine_back(MoveCall c)
{
    constexpr int PER = 256 / G;
    // (the same for all of a wave where a choice has one)
    const uint32_t sub = G == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / G) : threadIdx.x / G;
    const uint32_t f = (uint32_t)block_at() * PER + sub, all = (uint32_t)c.T * c.k;
    if (f >= all)
        return;
    const int lane = threadIdx.x % G;
    const int64_t t = f / (uint32_t)c.k;
    const int p = c.place[f];
    const bool none = p >= *c.n_rows, there = (uint32_t)p < all;
    const float w = c.weight ? c.weight[f] : 1.f;
    const typename O::raw *dout = (const typename O::raw *)c.dout + t * c.lddout;
    const typename E::raw *y = (const typename E::raw *)c.rows + (there ? p : 0) * c.ldrows;
    typename E::raw *dr = (typename E::raw *)c.drows + (there ? p : 0) * c.lddrows;
    const bool dots = c.dweight && !none && there;
    double dot = 0.0;
    for (int64_t c0 = 0; c0 < c.d; c0 += G * 8) {
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
        if constexpr (G == 64) {
            dot = wave_sum_f64(dot);
        } else {
#pragma unroll
            for (int o = 1; o < G; o <<= 1)
                dot += __shfl_xor(dot, o, 64);
        }
        if (lane == 0)
            c.dweight[f] = dots ? (float)dot : 0.f;
    }
}

// f(shift) for the threads per token: 8, 32 or 256, enough for a narrow row's chunks of eight.
template <class F>
void with_shift(int d, F f)
{
    if (d <= 64)
        f(std::integral_constant<int, 3>{});
    else if (d <= 512)
        f(std::integral_constant<int, 5>{});
    else
        f(std::integral_constant<int, 8>{});
}

dim3 token_grid(const MoveCall &c, int shift)
{
    const int per = 256 >> shift, cols = 8 << shift;
    return dim3((unsigned)((c.T + per - 1) / per), (unsigned)((c.d + cols - 1) / cols));
}

}  // namespace

int launch_token_sort(const SortCall &c, hipStream_t st)
{
    ProfScope prof("token_sort", st);
    const uint32_t rows = (uint32_t)c.T * c.k;
    const int n = sort_segments(rows);
    const uint32_t per = ((rows + n - 1) / n + kSortRows - 1) / kSortRows * kSortRows;  // whole steps of a block
    const size_t sh = (size_t)(c.E + 1) * 4;
    int bits = 0;
    while ((1 << bits) <= c.E)
        ++bits;
    if (rows <= 256 && c.E <= 256) {
        hipLaunchKernelGGL((k_token_place<4, true, true>), dim3(1), dim3(256), 6 * sh, st, c, 256, 1, bits);
    } else if (sort_counts_itself(n)) {
        hipLaunchKernelGGL((k_token_place<16, true, true>), dim3(n), dim3(1024), 18 * sh, st, c, kSortRows, n, bits);
    } else {
        hipLaunchKernelGGL(k_token_count, dim3(n), dim3(1024), sh, st, c, per);
        if (per == kSortRows)
            hipLaunchKernelGGL((k_token_place<16, true, false>), dim3(n), dim3(1024), 16 * sh, st, c, per, n, bits);
        else
            hipLaunchKernelGGL((k_token_place<16, false, false>), dim3(n), dim3(1024), 16 * sh, st, c, per, n, bits);
    }
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_dispatch(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_dispatch", st);
    with_element(c.dtype, [&](auto e) {
        with_bool(c.d % 8 == 0, [&](auto full) {
            with_shift(c.d, [&](auto shift) {
                using E = decltype(e);
                constexpr bool FULL = decltype(full)::value;
                constexpr int S = decltype(shift)::value;
                if (c.token_dtype == ECF_MXFP8)
                    hipLaunchKernelGGL((k_dispatch<E, true, FULL, S>), token_grid(c, S), dim3(256), 0, st, c);
                else
                    hipLaunchKernelGGL((k_dispatch<E, false, FULL, S>), token_grid(c, S), dim3(256), 0, st, c);
            });
        });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_combine_tokens(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_combine", st);
    with_pair(c.dtype, c.token_dtype, [&](auto e, auto o) {
        with_bool(c.d % 8 == 0, [&](auto full) {
            with_shift(c.d, [&](auto shift) {
                using E = decltype(e);
                using O = decltype(o);
                constexpr bool FULL = decltype(full)::value;
                constexpr int S = decltype(shift)::value;
#define ECF_COMBINE(KN) hipLaunchKernelGGL((k_combine_tokens<E, O, FULL, S, KN>), token_grid(c, S), dim3(256), 0, st, c)
                switch (c.k) {
                case 1: ECF_COMBINE(1); break;
                case 2: ECF_COMBINE(2); break;
                case 3: ECF_COMBINE(3); break;
                case 4: ECF_COMBINE(4); break;
                case 5: ECF_COMBINE(5); break;
                case 6: ECF_COMBINE(6); break;
                case 7: ECF_COMBINE(7); break;
                default: ECF_COMBINE(8);
                }
#undef ECF_COMBINE
            });
        });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

int launch_combine_backward(const MoveCall &c, hipStream_t st)
{
    ProfScope prof("token_combine_backward", st);
    // a wave per choice, or 8 or 32 lanes where they hold its row
    with_pair(c.dtype, c.token_dtype, [&](auto e, auto o) {
        with_bool(c.d % 8 == 0, [&](auto full) {
            using E = decltype(e);
            using O = decltype(o);
            constexpr bool FULL = decltype(full)::value;
            const auto grid = [&](int g) { return dim_of(block_grid(((int64_t)c.T * c.k * g + 255) / 256)); };
            if (c.d <= 64)
                hipLaunchKernelGGL((k_combine_back<E, O, FULL, 8>), grid(8), dim3(256), 0, st, c);
            else if (c.d <= 256)
                hipLaunchKernelGGL((k_combine_back<E, O, FULL, 32>), grid(32), dim3(256), 0, st, c);
            else
                hipLaunchKernelGGL((k_combine_back<E, O, FULL, 64>), grid(64), dim3(256), 0, st, c);
        });
    });
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

}  // namespace ecf
