// The token operators' internal interface: tokens.cpp and adapters.cpp check a call
// and carve its workspace, the launchers of k_norm.hip, k_tokens.hip and
// k_adapters.hip run it.
#pragma once

#include "arg_checks.h"
#include "ecf_internal.h"

namespace ecf {

constexpr int32_t kTokenMax = 1 << 22;  // tokens and widths per call
constexpr int kTileRows = 64;           // rows per tile of the sorted order

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
    float *partial;  // [norm_partial_rows(T)][d]
};
// Rows of column sums that the blocks of a backward pass leave behind for the weight's gradient.
int norm_partial_rows(int T);
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
// Segments of the choices that blocks of their own count and place (1: one block does all).
int sort_segments(int64_t rows);
inline size_t sort_ws(int64_t rows, int E)
{
    const int s = sort_segments(rows);
    return s > 1 ? al256((size_t)s * (E + 1) * 4) : 0;
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

}  // namespace ecf
