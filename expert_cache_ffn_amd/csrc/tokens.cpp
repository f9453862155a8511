// C-ABI entry points of the norm and of the tokens' way to experts and back:
// argument checks and workspaces.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "tokens_internal.h"

namespace ecf {
namespace {

constexpr int32_t kMaxExperts = 1024, kMaxTopK = 32;
constexpr int kNormParts = 512;  // rows of partial column sums, as far as there are tokens
// Segments up to which each block counts the others' choices itself, against a kernel that counts and one that
// places.  us a call in a graph, of 8 / 60 / 256 / 1024 experts: 5 segments 6.3 / 6.3 / 6.9 / 8.5 against 7.3 / 8.1 /
// 8.5 / 10.3; 8 segments 7.3 / 6.8 / 7.3 / 9.0 against 7.9 / 9.2 / 9.8 / 11.5; 16 segments 9.3 / 8.7 / 9.3 / 11.0
// against 8.1 / 8.6 / 9.3 / 11.0; 32 segments 13.7 / 12.7 / 13.2 / 15.1 against 9.9 / 11.0 / 11.4 / 13.4.
constexpr int kSortSelf = 8;
constexpr int kSortSegments = 128;  // most segments

int check_width(const char *what, int32_t d, int32_t T)
{
    if (d < 1 || d > kTokenMax || T < 0 || T > kTokenMax)
        return set_error(ECF_EINVAL, "%s: the width must be 1..%d and n_tokens 0..%d (d=%d, T=%d)", what, kTokenMax, kTokenMax,
                         d, T);
    return ECF_OK;
}

int check_norm(const char *what, const ecf_norm_args *a, int32_t T)
{
    if (!a)
        return set_error(ECF_EINVAL, "%s: args is NULL", what);
    ECF_TRY(check_width(what, a->hidden, T));
    if (!dense_dtype(a->dtype))
        return set_error(ECF_EINVAL, "%s: dtype must be ECF_F32, ECF_BF16 or ECF_F16 (got %d)", what, a->dtype);
    if (a->sum_dtype != a->dtype && a->sum_dtype != ECF_F32)
        return set_error(ECF_EINVAL, "%s: sum_dtype must be dtype or ECF_F32 (got %d)", what, a->sum_dtype);
    if (a->weight_dtype != a->dtype && a->weight_dtype != ECF_F32)
        return set_error(ECF_EINVAL, "%s: weight_dtype must be dtype or ECF_F32 (got %d)", what, a->weight_dtype);
    if (!(a->eps >= 0.f) || std::isinf(a->eps))
        return set_error(ECF_EINVAL, "%s: eps must be finite and not negative", what);
    return check_vector(what, "d_weight", a->d_weight, a->weight_dtype);
}

NormCall norm_call(const ecf_norm_args *a, int32_t T)
{
    NormCall c{};
    c.T = T, c.d = a->hidden;
    c.dtype = a->dtype, c.sum_dtype = a->sum_dtype, c.weight_dtype = a->weight_dtype, c.grad_dtype = a->wgrad_dtype;
    c.eps = a->eps;
    c.weight = a->d_weight;
    const int64_t d = a->hidden;
    c.sum = a->d_sum, c.ldsum = ld_or(a->ld_sum, d);
    c.rstd = a->d_rstd;
    return c;
}

int check_sort_shape(const char *what, int32_t E, int32_t k, int32_t T)
{
    if (E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || T < 0 || T > kTokenMax || (int64_t)T * k > kMaxRows)
        return set_error(ECF_EINVAL, "%s: n_experts must be 1..%d, top_k 1..%d, n_tokens 0..%d and n_tokens * top_k at most 2^26 "
                         "(E=%d, k=%d, T=%d)", what, kMaxExperts, kMaxTopK, kTokenMax, E, k, T);
    return ECF_OK;
}

int check_move(const char *what, const ecf_token_args *a, int32_t T, bool mx)
{
    if (!a)
        return set_error(ECF_EINVAL, "%s: args is NULL", what);
    ECF_TRY(check_width(what, a->hidden, T));
    ECF_TRY(check_sort_shape(what, a->n_experts, a->top_k, T));
    if (!dense_dtype(a->dtype))
        return set_error(ECF_EINVAL, "%s: dtype must be ECF_F32, ECF_BF16 or ECF_F16 (got %d)", what, a->dtype);
    const int32_t other = mx ? ECF_MXFP8 : ECF_F32;
    if (a->token_dtype != a->dtype && a->token_dtype != other)
        return set_error(ECF_EINVAL, "%s: token_dtype must be dtype or %s (got %d)", what, mx ? "ECF_MXFP8" : "ECF_F32",
                         a->token_dtype);
    if (T == 0)
        return ECF_OK;
    ECF_TRY(check_present(what, "d_offsets", a->d_offsets, 4));
    ECF_TRY(check_present(what, "d_place", a->d_place, 4));
    return check_aligned(what, "d_weight", a->d_weight, 4);
}

MoveCall move_call(const ecf_token_args *a, int32_t T)
{
    MoveCall c{};
    const int64_t d = a->hidden;
    c.T = T, c.k = a->top_k, c.d = a->hidden, c.dtype = a->dtype, c.token_dtype = a->token_dtype;
    c.place = a->d_place, c.n_rows = a->d_offsets + a->n_experts;
    c.weight = a->d_weight;
    c.rows = a->d_rows, c.ldrows = ld_or(a->ld_rows, d);
    return c;
}

}  // namespace

// Twice as many for short rows of many tokens, whose groups of threads are small (8192 tokens in bf16: 1024 elements 27.6
// us with 512 parts, 22.4 with 1024, 24.7 with 2048; 4096 elements, 4096 tokens 51.6, 57.7, 62.5).
int norm_partial_rows(int T, int d)
{
    int parts = kNormParts;
    if (d <= 2048 && T / 8 > parts)
        parts = T / 8 < 2 * kNormParts ? T / 8 : 2 * kNormParts;
    return T < parts ? T : parts;
}

int sort_segments(int64_t rows)
{
    const int64_t n = rows > 0 ? (rows + kSortRows - 1) / kSortRows : 1;
    return (int)(n < kSortSegments ? n : kSortSegments);
}

bool sort_counts_itself(int segments) { return segments <= kSortSelf; }

}  // namespace ecf

using namespace ecf;

extern "C" {

size_t ecf_norm_workspace_bytes(int32_t hidden, int32_t n_tokens, int32_t backward)
{
    if (check_width("ecf_norm_workspace_bytes", hidden, n_tokens) != ECF_OK)
        return SIZE_MAX;
    return backward ? al256((size_t)norm_partial_rows(n_tokens, hidden) * hidden * 4) : 0;
}

int ecf_norm_forward(const ecf_norm_args *a, int32_t T)
{
    return guarded("ecf_norm_forward", [&]() -> int {
        const char *me = "ecf_norm_forward";
        ECF_TRY(check_norm(me, a, T));
        if (T == 0)
            return ECF_OK;
        const int64_t d = a->hidden;
        NormCall c = norm_call(a, T);
        c.x = a->d_x, c.residual = a->d_residual;
        c.ldx = ld_or(a->ld_x, d), c.ldres = ld_or(a->ld_residual, d);
        c.y = a->d_y, c.ldy = ld_or(a->ld_y, d);
        c.q = a->d_q, c.ldq = ld_or(a->ld_q, d);
        c.q_scale = a->d_q_scale, c.ldqs = ld_or(a->ld_q_scale, (d + 31) / 32);
        ECF_TRY(check_rows(me, "d_x", c.x, c.ldx, d, a->dtype));
        if (c.residual)
            ECF_TRY(check_rows(me, "d_residual", c.residual, c.ldres, d, a->sum_dtype));
        else if (c.sum)
            return set_error(ECF_EINVAL, "%s: d_sum without d_residual (the sum is x)", me);
        if (c.sum)
            ECF_TRY(check_rows(me, "d_sum", c.sum, c.ldsum, d, a->sum_dtype));
        if (!c.y && !c.q)
            return set_error(ECF_EINVAL, "%s: neither d_y nor d_q is given", me);
        if (c.y)
            ECF_TRY(check_rows(me, "d_y", c.y, c.ldy, d, a->dtype));
        if (!c.q != !c.q_scale)
            return set_error(ECF_EINVAL, "%s: d_q and d_q_scale come together", me);
        if (c.q) {
            ECF_TRY(check_rows(me, "d_q", c.q, c.ldq, d, (size_t)1));
            ECF_TRY(check_rows(me, "d_q_scale", c.q_scale, c.ldqs, (d + 31) / 32, (size_t)1));
        }
        ECF_TRY(check_aligned(me, "d_rstd", c.rstd, 4));
        ECF_TRY(check_apart(me, {{"d_sum", c.sum}, {"d_y", c.y}, {"d_q", c.q}, {"d_q_scale", c.q_scale}, {"d_rstd", c.rstd}},
                            {{"d_x", c.x}, {"d_weight", c.weight}}));
        ECF_TRY(check_apart(me, {{"d_y", c.y}, {"d_q", c.q}, {"d_q_scale", c.q_scale}, {"d_rstd", c.rstd}},
                            {{"d_residual", c.residual}}));
        ECF_TRY(check_same_stride(me, "d_sum", c.sum, c.ldsum, "d_residual", c.residual, c.ldres));
        return launch_norm_forward(c, (hipStream_t)a->stream);
    });
}

int ecf_norm_backward(const ecf_norm_args *a, int32_t T)
{
    return guarded("ecf_norm_backward", [&]() -> int {
        const char *me = "ecf_norm_backward";
        ECF_TRY(check_norm(me, a, T));
        if (a->wgrad_dtype != a->weight_dtype && a->wgrad_dtype != ECF_F32)
            return set_error(ECF_EINVAL, "%s: wgrad_dtype must be weight_dtype or ECF_F32 (got %d)", me, a->wgrad_dtype);
        const int64_t d = a->hidden;
        NormCall c = norm_call(a, T);
        c.dy = a->d_dy, c.lddy = ld_or(a->ld_dy, d);
        c.dsum = a->d_dsum, c.lddsum = ld_or(a->ld_dsum, d);
        c.dx = a->d_dx, c.lddx = ld_or(a->ld_dx, d);
        c.ds = a->d_ds, c.ldds = ld_or(a->ld_ds, d);
        c.dweight = a->d_dweight;
        ECF_TRY(check_vector(me, "d_dweight", c.dweight, a->wgrad_dtype));
        if (T > 0) {
            ECF_TRY(check_rows(me, "d_sum", c.sum, c.ldsum, d, a->sum_dtype));
            ECF_TRY(check_present(me, "d_rstd", c.rstd, 4));
            ECF_TRY(check_rows(me, "d_dy", c.dy, c.lddy, d, a->dtype));
            if (c.dsum)
                ECF_TRY(check_rows(me, "d_dsum", c.dsum, c.lddsum, d, a->sum_dtype));
            if (c.dx)
                ECF_TRY(check_rows(me, "d_dx", c.dx, c.lddx, d, a->dtype));
            if (c.ds)
                ECF_TRY(check_rows(me, "d_ds", c.ds, c.ldds, d, a->sum_dtype));
        }
        const size_t need = c.dweight ? ecf_norm_workspace_bytes(a->hidden, T, 1) : 0;
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, need));
        ECF_TRY(check_apart(me, {{"d_dx", c.dx}, {"d_ds", c.ds}, {"d_dweight", c.dweight}, {"d_ws", need ? a->d_ws : nullptr}},
                            {{"d_sum", c.sum}, {"d_rstd", c.rstd}, {"d_dy", c.dy}, {"d_weight", c.weight}}));
        ECF_TRY(check_apart(me, {{"d_dx", c.dx}, {"d_dweight", c.dweight}, {"d_ws", need ? a->d_ws : nullptr}},
                            {{"d_dsum", c.dsum}}));
        ECF_TRY(check_same_stride(me, "d_ds", c.ds, c.ldds, "d_dsum", c.dsum, c.lddsum));
        c.partial = (float *)a->d_ws;
        return launch_norm_backward(c, (hipStream_t)a->stream);
    });
}

size_t ecf_token_sort_workspace_bytes(int32_t n_experts, int32_t top_k, int32_t n_tokens)
{
    if (check_sort_shape("ecf_token_sort_workspace_bytes", n_experts, top_k, n_tokens) != ECF_OK)
        return SIZE_MAX;
    return sort_ws((int64_t)n_tokens * top_k, n_experts);
}

int ecf_token_sort(const ecf_sort_args *a, int32_t T)
{
    return guarded("ecf_token_sort", [&]() -> int {
        const char *me = "ecf_token_sort";
        if (!a)
            return set_error(ECF_EINVAL, "%s: args is NULL", me);
        ECF_TRY(check_sort_shape(me, a->n_experts, a->top_k, T));
        if (a->idx_bytes != 4 && a->idx_bytes != 8)
            return set_error(ECF_EINVAL, "%s: idx_bytes must be 4 or 8 (got %d)", me, a->idx_bytes);
        SortCall c{};
        c.T = T, c.k = a->top_k, c.E = a->n_experts, c.wide = a->idx_bytes == 8;
        c.idx = a->d_idx, c.ldidx = ld_or(a->ld_idx, a->top_k);
        c.counts = a->d_counts, c.offsets = a->d_offsets, c.tiles = a->d_tiles, c.order = a->d_order, c.place = a->d_place;
        ECF_TRY(check_present(me, "d_counts", c.counts, 4));
        ECF_TRY(check_present(me, "d_offsets", c.offsets, 4));
        ECF_TRY(check_present(me, "d_tiles", c.tiles, 4));
        if (T > 0) {
            ECF_TRY(check_rows(me, "d_idx", c.idx, c.ldidx, a->top_k, (size_t)a->idx_bytes));
            ECF_TRY(check_present(me, "d_order", c.order, 4));
            ECF_TRY(check_present(me, "d_place", c.place, 4));
        } else {
            c.idx = nullptr, c.order = c.place = nullptr;  // of no length
        }
        const size_t need = sort_ws((int64_t)T * a->top_k, a->n_experts);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, need));
        c.segments = (int32_t *)a->d_ws;
        ECF_TRY(check_apart(me, {{"d_counts", c.counts}, {"d_offsets", c.offsets}, {"d_tiles", c.tiles}, {"d_order", c.order},
                                 {"d_place", c.place}, {"d_ws", need ? a->d_ws : nullptr}}, {{"d_idx", c.idx}}));
        return launch_token_sort(c, (hipStream_t)a->stream);
    });
}

int ecf_token_dispatch(const ecf_token_args *a, int32_t T)
{
    return guarded("ecf_token_dispatch", [&]() -> int {
        const char *me = "ecf_token_dispatch";
        ECF_TRY(check_move(me, a, T, true));
        if (T == 0)
            return ECF_OK;
        const int64_t d = a->hidden;
        MoveCall c = move_call(a, T);
        const bool mx = a->token_dtype == ECF_MXFP8;
        c.x = a->d_x, c.ldx = ld_or(a->ld_x, d);
        c.x_scale = a->d_x_scale, c.ldxs = ld_or(a->ld_x_scale, (d + 31) / 32);
        ECF_TRY(check_rows(me, "d_x", c.x, c.ldx, d, mx ? (size_t)1 : dense_esize(a->dtype)));
        if (mx)
            ECF_TRY(check_rows(me, "d_x_scale", c.x_scale, c.ldxs, (d + 31) / 32, (size_t)1));
        ECF_TRY(check_rows(me, "d_rows", c.rows, c.ldrows, d, a->dtype));
        ECF_TRY(check_apart(me, {{"d_rows", c.rows}}, {{"d_x", c.x}, {"d_x_scale", mx ? c.x_scale : nullptr},
                                                       {"d_offsets", a->d_offsets}, {"d_place", c.place}}));
        return launch_dispatch(c, (hipStream_t)a->stream);
    });
}

int ecf_token_combine(const ecf_token_args *a, int32_t T)
{
    return guarded("ecf_token_combine", [&]() -> int {
        const char *me = "ecf_token_combine";
        ECF_TRY(check_move(me, a, T, false));
        if (T == 0)
            return ECF_OK;
        const int64_t d = a->hidden;
        MoveCall c = move_call(a, T);
        c.residual = a->d_residual, c.ldres = ld_or(a->ld_residual, d);
        c.out = a->d_out, c.ldout = ld_or(a->ld_out, d);
        ECF_TRY(check_rows(me, "d_rows", c.rows, c.ldrows, d, a->dtype));
        ECF_TRY(check_rows(me, "d_out", c.out, c.ldout, d, a->token_dtype));
        if (c.residual)
            ECF_TRY(check_rows(me, "d_residual", c.residual, c.ldres, d, a->token_dtype));
        ECF_TRY(check_apart(me, {{"d_out", c.out}}, {{"d_rows", c.rows}, {"d_offsets", a->d_offsets}, {"d_place", c.place},
                                                     {"d_weight", c.weight}}));
        ECF_TRY(check_same_stride(me, "d_out", c.out, c.ldout, "d_residual", c.residual, c.ldres));
        return launch_combine_tokens(c, (hipStream_t)a->stream);
    });
}

int ecf_token_combine_backward(const ecf_token_args *a, int32_t T)
{
    return guarded("ecf_token_combine_backward", [&]() -> int {
        const char *me = "ecf_token_combine_backward";
        ECF_TRY(check_move(me, a, T, false));
        if (T == 0)
            return ECF_OK;
        const int64_t d = a->hidden;
        MoveCall c = move_call(a, T);
        c.dout = a->d_dout, c.lddout = ld_or(a->ld_dout, d);
        c.drows = a->d_drows, c.lddrows = ld_or(a->ld_drows, d);
        c.dweight = a->d_dweight;
        if (!c.drows && !c.dweight)
            return ECF_OK;
        ECF_TRY(check_rows(me, "d_dout", c.dout, c.lddout, d, a->token_dtype));
        if (c.dweight)
            ECF_TRY(check_rows(me, "d_rows", c.rows, c.ldrows, d, a->dtype));
        if (c.drows)
            ECF_TRY(check_rows(me, "d_drows", c.drows, c.lddrows, d, a->dtype));
        ECF_TRY(check_aligned(me, "d_dweight", c.dweight, 4));
        ECF_TRY(check_apart(me, {{"d_drows", c.drows}, {"d_dweight", c.dweight}},
                            {{"d_dout", c.dout}, {"d_rows", c.dweight ? c.rows : nullptr}, {"d_offsets", a->d_offsets},
                             {"d_place", c.place}, {"d_weight", c.weight}}));
        return launch_combine_backward(c, (hipStream_t)a->stream);
    });
}

}  // extern "C"
