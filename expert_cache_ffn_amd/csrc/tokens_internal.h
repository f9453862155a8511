// The token operators' internal interface: tokens.cpp and adapters.cpp check a call
// and carve its workspace, the launchers of k_norm.hip, k_tokens.hip and
// k_adapters.hip run it.
#pragma once

#include "arg_checks.h"
#include "ecf_internal.h"

namespace ecf {

constexpr int32_t kTokenMax = 1 << 22;  // tokens and widths per call
constexpr int kTileRows = 64;           // rows per tile of the sorted order

// One dimension of a grid takes fewer than 2^32 threads.  Where there may be more, with up to 1024 a block, block b is
// (b % kGridX, b / kGridX); those behind the last one, which complete the last line, return.
constexpr int kGridX = 1 << 21;
struct BlockGrid {
    unsigned x, y;
};
inline BlockGrid block_grid(int64_t blocks)
{
    return {(unsigned)(blocks < kGridX ? blocks : kGridX), (unsigned)((blocks + kGridX - 1) / kGridX)};
}

// ---- norm ---------------------------------------------------------------------------
struct NormCall {
    int T, d, dtype, sum_dtype, weight_dtype, grad_dtype;
    float eps;
    const void *weight;  // null: ones
    // forward
    const void *x, *residual;
    int64_t ldx, ldres;
    void *sum, *y, *q, *q_scale;
    int64_t ldsum, ldy, ldq, ldqs;
    float *rstd;
    // backward (reads sum and rstd)
    const void *dy, *dsum;
    int64_t lddy, lddsum;
    void *dx, *ds;
    int64_t lddx, ldds;
    void *dweight;
    float *partial;  // [norm_partial_rows(T, d)][d]
};
// Rows of column sums that the blocks of a backward pass leave behind for the weight's gradient.
int norm_partial_rows(int T, int d);
int launch_norm_forward(const NormCall &c, hipStream_t st);
int launch_norm_backward(const NormCall &c, hipStream_t st);

// ---- tokens by expert ------------------------------------------------------------------
struct SortCall {
    int T, k, E, wide;  // wide: 64-bit ids
    const void *idx;
    int64_t ldidx;
    int32_t *counts, *offsets, *tiles, *order, *place;
    int32_t *segments;  // workspace: [sort_segments][E + 1]
};
constexpr int kSortRows = 1024;  // choices that a block takes at a time
// Segments of the choices, which blocks of their own place; many have their counts in the workspace.
int sort_segments(int64_t rows);
bool sort_counts_itself(int segments);
inline size_t sort_ws(int64_t rows, int E)
{
    const int s = sort_segments(rows);
    return sort_counts_itself(s) ? 0 : al256((size_t)s * (E + 1) * 4);
}
int launch_token_sort(const SortCall &c, hipStream_t st);

struct MoveCall {
    int T, k, d, dtype, token_dtype;
    const int32_t *place;
    const int32_t *n_rows;  // rows of any expert (offsets + E)
    const float *weight;
    const void *x, *x_scale;
    int64_t ldx, ldxs;
    void *rows;
    int64_t ldrows;
    const void *residual;
    int64_t ldres;
    void *out;
    int64_t ldout;
    const void *dout;
    int64_t lddout;
    void *drows;
    int64_t lddrows;
    float *dweight;
};
int launch_dispatch(const MoveCall &c, hipStream_t st);
int launch_combine_tokens(const MoveCall &c, hipStream_t st);
int launch_combine_backward(const MoveCall &c, hipStream_t st);

// ---- low-rank adapters -------------------------------------------------------------------
// The sorted order of the tokens' adapters.
struct AdapterOrder {
    const void *idx;
    int wide;  // 64-bit ids
    const int32_t *order, *offsets, *tiles;
    int T, n;
};
// Tokens up to which a forward pass takes them one by one, without an order.
constexpr int kAdapterFew = 64;

// part[s][t][j] = sum over split s of k of x[t][k] M[a](j, k): A[a] as it lies, [r][K] (of_b
// false), or B[a]'s transpose (of_b: M[a] lies as [K][r]); t the row of the order, where there is one.
struct ShrinkCall {
    AdapterOrder o;
    int dtype, x_dtype, K, r;
    bool of_b;
    const void *m, *x;
    int64_t ldx;
    float *part;
    int splits, split_k;  // split_k: k per split, a multiple of kShrinkChunk
};
// Most splits by 72 tiles of 64 tokens, K 4096: 12.1 us, 13.5 with 8, 24 with 2 (fewer tiles were not measured with more).
constexpr int kShrinkBlocks = 1024, kShrinkSplits = 7;
constexpr int kShrinkChunk = 128;  // k that a block stages at a time
int shrink_split_k(int T, int K);
int shrink_splits(int T, int K);
// Rows of h in all splits of any call of up to T tokens.
inline int64_t shrink_rows(int64_t T)
{
    const int64_t split = kShrinkSplits * T < kShrinkBlocks * kTileRows ? kShrinkSplits * T : kShrinkBlocks * kTileRows;
    return split > T ? split : T;
}
int launch_shrink(const ShrinkCall &c, hipStream_t st);

// h[t][j] = sum of the splits, out[t][i] = residual[t][i] + scale[a] * sum_j h[t][j] M[a](i, j):
// B[a] as it lies, [N][r], or A[a]'s transpose (of_a: M[a] lies as [r][N]).
struct ExpandCall {
    AdapterOrder o;
    int dtype, out_dtype, N, r;
    bool of_a;
    const void *m;
    const float *scale;  // null: ones
    const float *part;
    int splits;
    float *h;          // [T][r], written; or null
    bool scaled;       // h is written times the scale
    const void *residual;
    int64_t ldres;
    void *out;  // null: h only
    int64_t ldout;
};
int launch_expand(const ExpandCall &c, hipStream_t st);

// Few tokens, in any order: both in one launch, without a workspace, or with h between two kernels.
constexpr int kFewCols = 1024;                // columns per block of the one
// Of a token's A, which each of its blocks reads, counted in fp32 for all types (the size query does not know it).
// us a call in a graph, in one launch / in two, 16 tokens, K to K: bf16 rank 16 of 2048 4.4 / 5.5, 32 of 2048 6.2 / 6.3, 16 of
// 4096 5.4 / 5.9 (64 tokens 8.6 / 7.4), 24 of 4096 6.6 / 6.3, 16 of 8192 10.9 / 6.8; fp32, whose own border is half as
// far, rank 16 of 2048 5.4 / 5.8, 8 of 4096 5.2 / 5.5, 16 of 4096 7.2 / 6.2, 32 of 2048 9.9 / 6.7.
constexpr int64_t kFewBytes = (int64_t)1 << 18;
inline bool adapter_few_in_one(int64_t T, int64_t K, int64_t N, int64_t r, int esize)
{
    return T <= kAdapterFew && T * ((N + kFewCols - 1) / kFewCols) <= 256 && r * K * esize <= kFewBytes;
}
int launch_few(const ShrinkCall &c, const ExpandCall &x, hipStream_t st);
int launch_few_shrink(const ShrinkCall &c, hipStream_t st);
int launch_few_expand(const ExpandCall &c, hipStream_t st);

// d[a](j, i) = sum over a's tokens of g[t][j] * gscale[a] * x[t][i], as [r][W] (dA) or [W][r] (dB)
struct OuterCall {
    AdapterOrder o;
    int x_dtype, grad_dtype, W, r;
    bool of_b;
    const float *g;
    const float *gscale;  // null: ones
    const void *x;
    int64_t ldx;
    void *d;
    float *slots;  // outer_slots bytes
};
constexpr int kOuterCols = 128;  // columns per block
int outer_slices(int W);
// Runs of the sorted rows, blocks of their own, for so many slices of columns.
int outer_chunks(int T, int slices);
inline size_t outer_slots(int chunks, int W, int r) { return chunks > 1 ? al256((size_t)chunks * 2 * W * r * 4) : 0; }
// One or two of one rank and x_dtype over the same order.
int launch_outer(const OuterCall *calls, int n, int chunks, hipStream_t st);

}  // namespace ecf
