// C-ABI entry points of the dense feed-forward operators: argument checks, the
// workspace, and the matrix products and gradient kernels each call is made of.
#include <algorithm>
#include <cstdint>

#include "arg_checks.h"
#include "dense_internal.h"

namespace ecf {
namespace {

constexpr int32_t kDenseMax = 1 << 22;  // tokens and widths per call

int check_common(const char *what, int32_t in, int32_t out, int32_t dtype, int32_t T)
{
    if (in < 1 || in > kDenseMax || out < 1 || out > kDenseMax || T < 0 || T > kDenseMax)
        return set_error(ECF_EINVAL, "%s: widths must be 1..%d and n_tokens 0..%d (in=%d, out=%d, T=%d)", what,
                         kDenseMax, kDenseMax, in, out, T);
    if (!dense_dtype(dtype))
        return set_error(ECF_EINVAL, "%s: dtype must be ECF_F32, ECF_BF16 or ECF_F16 (got %d)", what, dtype);
    return ECF_OK;
}

// 256 rows lie within a 31-bit byte offset.
int64_t longest_row(int dtype) { return 0x7fffffff / 256 / (int64_t)dense_esize(dtype); }

// What a size query refuses: also widths that no call takes.
int check_query(const char *what, int32_t in, int32_t out, int32_t dtype, int32_t T)
{
    const int rc = check_common(what, in, out, dtype, T);
    if (rc == ECF_OK && T > 0 && std::max(in, out) > longest_row(dtype))
        return set_error(ECF_EUNSUPPORTED, "%s: 256 rows of %d elements span 2 GiB or more", what, std::max(in, out));
    return rc;
}

// A matrix operand: present, aligned to its element, rows at least as far apart
// as they are long, and 256 of them within a 31-bit byte offset.
int check_matrix(const char *what, const char *name, const void *p, int64_t ld, int64_t width, int dtype)
{
    const size_t e = dense_esize(dtype);
    if (!p)
        return set_error(ECF_EINVAL, "%s: %s is NULL", what, name);
    if ((uintptr_t)p % e)
        return set_error(ECF_EINVAL, "%s: %s is not aligned to its %zu-byte elements", what, name, e);
    if (ld < width)
        return set_error(ECF_EINVAL, "%s: the row stride of %s (%lld) is below its width %lld", what, name,
                         (long long)ld, (long long)width);
    if (ld > longest_row(dtype))
        return set_error(ECF_EUNSUPPORTED, "%s: 256 rows of %s (stride %lld) span 2 GiB or more", what, name,
                         (long long)ld);
    return ECF_OK;
}

int check_act(const char *what, int32_t act)
{
    if (act < ECF_ACT_NONE || act > ECF_ACT_RELU)
        return set_error(ECF_EINVAL, "%s: unknown activation %d", what, act);
    return ECF_OK;
}

// A few tokens' calls have no workspace: their weights are streamed, or (16-bit rows
// that start at odd elements) go through tiles that do not split K.  Rows of odd length
// always start so; there the split tiles may be the fastest.
size_t forward_ws(int64_t T, int64_t in, int64_t out, int dtype, int planes)
{
    return few_needs_no_room(T, in) && (dtype == ECF_F32 || in % 2 == 0) ? 0
               : dense_gemm_ws(T, out, in, 1, planes);
}

// Backward workspace: dz rows in `dtype` (gated: all of da, then all of db), at 16-byte
// boundaries (rows of dh or dy rounded up to 8 elements, so the last of 256 starts and
// ends within a 31-bit byte offset as theirs does), the column sums of each row block in
// fp32, the products' partial sums, and for a scaled fp16 pass (DenseGrad) a second dz,
// what the scales are found from and their inverses.
struct BackWs {
    int64_t pitch;
    size_t split, room, dz, dz_w, row_tops, col_tops, row_inverse, col_inverse, total;  // the column sums start it
};
BackWs back_ws(int64_t in, int64_t cols, int halves, int dtype, int32_t T, bool dz = true)
{
    BackWs w{};
    const size_t row_blocks = (size_t)dense_grad_max_row_blocks(T);
    w.pitch = (cols + 7) / 8 * 8;
    w.split = al256(row_blocks * halves * cols * 4);
    // both products' in one launch, or either's in turn
    w.room = std::min(dense_gemm_ws(T, in, cols, halves, 1) + dense_gemm_ws(cols, in, T, 1, halves), kDensePartialBytes);
    w.dz = w.total = w.split + w.room;
    if (!dz)
        return w;
    const size_t plane = al256((size_t)T * w.pitch * halves * dense_esize(dtype));
    w.dz_w = w.total = w.dz + plane;
    if (dtype != ECF_F16)
        return w;
    w.row_tops = w.dz_w + plane;
    w.col_tops = w.row_tops + al256((size_t)dense_grad_col_blocks(cols) * T * 4);
    w.row_inverse = w.col_tops + al256(row_blocks * halves * cols * 4);
    w.col_inverse = w.row_inverse + al256((size_t)T * 4);
    w.total = w.col_inverse + al256((size_t)halves * cols * 4);
    return w;
}

// What of dz a backward pass writes, for the products that are wanted: one for both, or (scaled) one each.
void set_dz(DenseGrad &q, const BackWs &w, char *ws, bool dx, bool dw, bool scaled)
{
    q.pitch = w.pitch;
    q.scaled = scaled && (dx || dw);
    q.dz = dx || (dw && !q.scaled) ? ws + w.dz : nullptr;
    if (!q.scaled)
        return;
    q.dz_w = dw ? ws + w.dz_w : nullptr;
    q.row_tops = (uint32_t *)(ws + w.row_tops), q.col_tops = (uint32_t *)(ws + w.col_tops);
    q.row_inverse = (float *)(ws + w.row_inverse), q.col_inverse = (float *)(ws + w.col_inverse);
}

}  // namespace
}  // namespace ecf

using namespace ecf;

extern "C" {

size_t ecf_gated_workspace_bytes(int32_t hidden, int32_t inter, int32_t dtype, int32_t n_tokens, int32_t backward)
{
    if (check_query("ecf_gated_workspace_bytes", hidden, inter, dtype, n_tokens) != ECF_OK)
        return SIZE_MAX;
    return backward ? back_ws(hidden, inter, 2, dtype, n_tokens).total : forward_ws(n_tokens, hidden, inter, dtype, 2);
}

int ecf_gated_forward(const ecf_gated_args *a, int32_t T)
{
    return guarded("ecf_gated_forward", [&]() -> int {
        const char *me = "ecf_gated_forward";
        if (!a)
            return set_error(ECF_EINVAL, "%s: args is NULL", me);
        ECF_TRY(check_common(me, a->hidden, a->inter, a->dtype, T));
        ECF_TRY(check_act(me, a->act));
        const int64_t d = a->hidden, I = a->inter;
        DenseGemm g{};
        g.dtype = g.out_dtype = a->dtype;
        g.gated = true;
        g.ksegs = g.mhalves = 1;
        g.M = T, g.N = a->inter, g.K = a->hidden;
        g.lda = ld_or(a->ld_x, d), g.ldb = ld_or(a->ld_w, d);
        g.ldout = ld_or(a->ld_h, I), g.ldsave = ld_or(a->ld_ab, I);
        g.act = a->act;
        if (T == 0)
            return ECF_OK;
        ECF_TRY(check_matrix(me, "d_x", a->d_x, g.lda, d, a->dtype));
        ECF_TRY(check_matrix(me, "d_w_gate", a->d_w_gate, g.ldb, d, a->dtype));
        ECF_TRY(check_matrix(me, "d_w_up", a->d_w_up, g.ldb, d, a->dtype));
        ECF_TRY(check_vector(me, "d_b_gate", a->d_b_gate, a->dtype));
        ECF_TRY(check_vector(me, "d_b_up", a->d_b_up, a->dtype));
        if (!a->d_a != !a->d_b)
            return set_error(ECF_EINVAL, "%s: d_a and d_b come together", me);
        if (a->d_h || !a->d_a)
            ECF_TRY(check_matrix(me, "d_h", a->d_h, g.ldout, I, a->dtype));
        if (a->d_a) {
            ECF_TRY(check_matrix(me, "d_a", a->d_a, g.ldsave, I, a->dtype));
            ECF_TRY(check_matrix(me, "d_b", a->d_b, g.ldsave, I, a->dtype));
        }
        const size_t need = forward_ws(T, d, I, a->dtype, 2);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, need));
        ECF_TRY(check_apart(me, {{"d_h", a->d_h}, {"d_a", a->d_a}, {"d_b", a->d_b}, {"d_ws", need ? a->d_ws : nullptr}},
                              {{"d_x", a->d_x}, {"d_w_gate", a->d_w_gate}, {"d_w_up", a->d_w_up},
                               {"d_b_gate", a->d_b_gate}, {"d_b_up", a->d_b_up}}));
        g.a[0] = a->d_x;
        g.b[0] = a->d_w_gate, g.b[1] = a->d_w_up;
        g.bias[0] = a->d_b_gate, g.bias[1] = a->d_b_up;
        g.out[0] = a->d_h;
        g.save[0] = a->d_a, g.save[1] = a->d_b;
        return launch_dense_gemm(g, need ? a->d_ws : nullptr, need, (hipStream_t)a->stream);
    });
}

int ecf_gated_backward(const ecf_gated_args *a, int32_t T)
{
    return guarded("ecf_gated_backward", [&]() -> int {
        const char *me = "ecf_gated_backward";
        if (!a)
            return set_error(ECF_EINVAL, "%s: args is NULL", me);
        ECF_TRY(check_common(me, a->hidden, a->inter, a->dtype, T));
        ECF_TRY(check_act(me, a->act));
        ECF_TRY(check_grad_dtype(me, a->wgrad_dtype, a->dtype));
        const int64_t d = a->hidden, I = a->inter;
        const int64_t ldx = ld_or(a->ld_x, d), ldw = ld_or(a->ld_w, d), ldab = ld_or(a->ld_ab, I),
                      lddh = ld_or(a->ld_dh, I), lddx = ld_or(a->ld_dx, d), lddw = ld_or(a->ld_dw, d);
        if (!a->d_dw_gate != !a->d_dw_up)
            return set_error(ECF_EINVAL, "%s: d_dw_gate and d_dw_up come together", me);
        const bool want_dw = a->d_dw_gate, want_db = a->d_db_gate || a->d_db_up, want_dx = a->d_dx && T > 0;
        if (T > 0) {
            ECF_TRY(check_matrix(me, "d_a", a->d_a, ldab, I, a->dtype));
            ECF_TRY(check_matrix(me, "d_b", a->d_b, ldab, I, a->dtype));
            ECF_TRY(check_matrix(me, "d_dh", a->d_dh, lddh, I, a->dtype));
            if (want_dw)
                ECF_TRY(check_matrix(me, "d_x", a->d_x, ldx, d, a->dtype));
        }
        if (want_dx) {
            ECF_TRY(check_matrix(me, "d_w_gate", a->d_w_gate, ldw, d, a->dtype));
            ECF_TRY(check_matrix(me, "d_w_up", a->d_w_up, ldw, d, a->dtype));
            ECF_TRY(check_matrix(me, "d_dx", a->d_dx, lddx, d, a->dtype));
        }
        if (want_dw) {
            ECF_TRY(check_matrix(me, "d_dw_gate", a->d_dw_gate, lddw, d, a->wgrad_dtype));
            ECF_TRY(check_matrix(me, "d_dw_up", a->d_dw_up, lddw, d, a->wgrad_dtype));
        }
        ECF_TRY(check_vector(me, "d_db_gate", a->d_db_gate, a->wgrad_dtype));
        ECF_TRY(check_vector(me, "d_db_up", a->d_db_up, a->wgrad_dtype));
        const BackWs w = back_ws(d, I, 2, a->dtype, T);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, w.total));
        ECF_TRY(check_apart(me, {{"d_dx", a->d_dx}, {"d_dw_gate", a->d_dw_gate}, {"d_dw_up", a->d_dw_up},
                                   {"d_db_gate", a->d_db_gate}, {"d_db_up", a->d_db_up}, {"d_ws", a->d_ws}},
                              {{"d_x", a->d_x}, {"d_w_gate", a->d_w_gate}, {"d_w_up", a->d_w_up}, {"d_a", a->d_a},
                               {"d_b", a->d_b}, {"d_dh", a->d_dh}}));
        hipStream_t st = (hipStream_t)a->stream;
        char *ws = (char *)a->d_ws;
        DenseColsum sums{};
        DenseGemm gx{}, gw{};
        if (want_db || (T > 0 && (want_dw || want_dx))) {
            DenseGrad q{};
            q.dtype = q.dout_dtype = a->dtype;
            q.act = a->act;
            q.gated = true;
            q.dout = a->d_dh, q.a = a->d_a, q.b = a->d_b;
            q.lddout = lddh, q.ldab = ldab;
            q.T = T, q.I = a->inter;
            set_dz(q, w, ws, want_dx, want_dw, a->dtype == ECF_F16 && T > 0);
            q.want_sums = want_db;
            q.sums[0] = a->d_db_gate, q.sums[1] = a->d_db_up;
            q.sums_dtype = a->wgrad_dtype;
            q.partial = (float *)ws;
            ECF_TRY(launch_dense_grad(q, &sums, st));
            gx.unscale = q.row_inverse, gw.unscale = q.col_inverse;
            gx.a[0] = q.dz, gw.a[0] = q.scaled ? q.dz_w : q.dz;
        }
        const size_t half = (size_t)T * w.pitch * dense_esize(a->dtype);
        gx.dtype = gx.out_dtype = gw.dtype = a->dtype;
        gx.b_t = gw.a_t = gw.b_t = true;
        gx.ksegs = gw.mhalves = 2;
        gx.mhalves = gw.ksegs = 1;
        gx.a[1] = (const char *)gx.a[0] + half, gw.a[1] = (const char *)gw.a[0] + half;
        gx.lda = gw.lda = w.pitch;
        gx.a_padded = gw.a_padded = true;
        gx.b[0] = a->d_w_gate, gx.b[1] = a->d_w_up;
        gx.ldb = ldw;
        gx.M = T, gx.N = a->hidden, gx.K = a->inter;
        gx.out[0] = a->d_dx;
        gx.ldout = lddx;
        gw.out_dtype = a->wgrad_dtype;
        gw.b[0] = a->d_x;
        gw.ldb = ldx;
        gw.M = a->inter, gw.N = a->hidden, gw.K = T;
        gw.out[0] = a->d_dw_gate, gw.out[1] = a->d_dw_up;
        gw.ldout = lddw;
        return launch_dense_backward(want_dx ? &gx : nullptr, want_dw ? &gw : nullptr, sums, ws + w.split, w.room, st);
    });
}

size_t ecf_linear_workspace_bytes(int32_t in_features, int32_t out_features, int32_t dtype, int32_t n_tokens,
                                  int32_t backward)
{
    if (check_query("ecf_linear_workspace_bytes", in_features, out_features, dtype, n_tokens) != ECF_OK)
        return SIZE_MAX;
    return backward ? back_ws(in_features, out_features, 1, dtype, n_tokens, backward != 2).total
                    : forward_ws(n_tokens, in_features, out_features, dtype, 1);
}

int ecf_linear_forward(const ecf_linear_args *a, int32_t T)
{
    return guarded("ecf_linear_forward", [&]() -> int {
        const char *me = "ecf_linear_forward";
        if (!a)
            return set_error(ECF_EINVAL, "%s: args is NULL", me);
        ECF_TRY(check_common(me, a->in_features, a->out_features, a->dtype, T));
        ECF_TRY(check_act(me, a->act));
        if (a->out_dtype != a->dtype && a->out_dtype != ECF_F32)
            return set_error(ECF_EINVAL, "%s: out_dtype must be dtype or ECF_F32 (got %d)", me, a->out_dtype);
        const int64_t K = a->in_features, N = a->out_features;
        DenseGemm g{};
        g.dtype = a->dtype, g.out_dtype = a->out_dtype;
        g.ksegs = g.mhalves = 1;
        g.M = T, g.N = a->out_features, g.K = a->in_features;
        g.lda = ld_or(a->ld_x, K), g.ldb = ld_or(a->ld_w, K);
        g.ldout = ld_or(a->ld_out, N), g.ldsave = ld_or(a->ld_z, N), g.ldres = ld_or(a->ld_residual, N);
        g.act = a->act;
        if (T == 0)
            return ECF_OK;
        ECF_TRY(check_matrix(me, "d_x", a->d_x, g.lda, K, a->dtype));
        ECF_TRY(check_matrix(me, "d_w", a->d_w, g.ldb, K, a->dtype));
        ECF_TRY(check_matrix(me, "d_out", a->d_out, g.ldout, N, a->out_dtype));
        ECF_TRY(check_vector(me, "d_bias", a->d_bias, a->dtype));
        if (a->d_residual)
            ECF_TRY(check_matrix(me, "d_residual", a->d_residual, g.ldres, N, a->out_dtype));
        if (a->d_z)
            ECF_TRY(check_matrix(me, "d_z", a->d_z, g.ldsave, N, a->dtype));
        const size_t need = forward_ws(T, K, N, a->dtype, 1);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, need));
        ECF_TRY(check_apart(me, {{"d_out", a->d_out}, {"d_z", a->d_z}, {"d_ws", need ? a->d_ws : nullptr}},
                              {{"d_x", a->d_x}, {"d_w", a->d_w}, {"d_bias", a->d_bias}}));
        ECF_TRY(check_apart(me, {{"d_z", a->d_z}, {"d_ws", need ? a->d_ws : nullptr}}, {{"d_residual", a->d_residual}}));
        if (a->d_out == a->d_residual && g.ldout != g.ldres)
            return set_error(ECF_EINVAL, "%s: d_out is d_residual with another row stride (%lld and %lld)", me,
                             (long long)g.ldout, (long long)g.ldres);
        g.a[0] = a->d_x, g.b[0] = a->d_w;
        g.bias[0] = a->d_bias;
        g.res = a->d_residual;
        g.out[0] = a->d_out;
        g.save[0] = a->d_z;
        return launch_dense_gemm(g, need ? a->d_ws : nullptr, need, (hipStream_t)a->stream);
    });
}

int ecf_linear_backward(const ecf_linear_args *a, int32_t T)
{
    return guarded("ecf_linear_backward", [&]() -> int {
        const char *me = "ecf_linear_backward";
        if (!a)
            return set_error(ECF_EINVAL, "%s: args is NULL", me);
        ECF_TRY(check_common(me, a->in_features, a->out_features, a->dtype, T));
        ECF_TRY(check_act(me, a->act));
        ECF_TRY(check_grad_dtype(me, a->wgrad_dtype, a->dtype));
        if (a->out_dtype != a->dtype && a->out_dtype != ECF_F32)
            return set_error(ECF_EINVAL, "%s: out_dtype must be dtype or ECF_F32 (got %d)", me, a->out_dtype);
        const int64_t K = a->in_features, N = a->out_features;
        const int64_t ldx = ld_or(a->ld_x, K), ldw = ld_or(a->ld_w, K), ldz = ld_or(a->ld_z, N),
                      lddy = ld_or(a->ld_dout, N), lddx = ld_or(a->ld_dx, K), lddw = ld_or(a->ld_dw, K);
        const bool want_dx = a->d_dx && T > 0, act = a->act != ECF_ACT_NONE;
        if (T > 0) {
            ECF_TRY(check_matrix(me, "d_dout", a->d_dout, lddy, N, a->out_dtype));
            if (act)
                ECF_TRY(check_matrix(me, "d_z", a->d_z, ldz, N, a->dtype));
            if (a->d_dw)
                ECF_TRY(check_matrix(me, "d_x", a->d_x, ldx, K, a->dtype));
        }
        if (want_dx) {
            ECF_TRY(check_matrix(me, "d_w", a->d_w, ldw, K, a->dtype));
            ECF_TRY(check_matrix(me, "d_dx", a->d_dx, lddx, K, a->dtype));
        }
        if (a->d_dw)
            ECF_TRY(check_matrix(me, "d_dw", a->d_dw, lddw, K, a->wgrad_dtype));
        ECF_TRY(check_vector(me, "d_dbias", a->d_dbias, a->wgrad_dtype));
        // without an activation and in the operands' type, dy is dz
        const bool direct = !act && a->out_dtype == a->dtype;
        const BackWs w = back_ws(K, N, 1, a->dtype, T, !direct);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, w.total));
        ECF_TRY(check_apart(me, {{"d_dx", a->d_dx}, {"d_dw", a->d_dw}, {"d_dbias", a->d_dbias}, {"d_ws", a->d_ws}},
                              {{"d_x", a->d_x}, {"d_w", a->d_w}, {"d_z", a->d_z}, {"d_dout", a->d_dout}}));
        hipStream_t st = (hipStream_t)a->stream;
        const bool products = want_dx || (a->d_dw && T > 0);
        DenseColsum sums{};
        DenseGemm gx{}, gw{};
        if (a->d_dbias || (T > 0 && products && !direct)) {
            DenseGrad q{};
            q.dtype = a->dtype, q.dout_dtype = a->out_dtype;
            q.act = a->act;
            q.dout = a->d_dout;
            q.a = act ? a->d_z : nullptr;
            q.lddout = lddy, q.ldab = ldz;
            q.T = T, q.I = a->out_features;
            // (relu leaves an fp16 dy what it is, or zero)
            if (products && !direct)
                set_dz(q, w, (char *)a->d_ws, want_dx, a->d_dw != nullptr,
                       a->dtype == ECF_F16 && !(a->act == ECF_ACT_RELU && a->out_dtype == ECF_F16));
            q.want_sums = a->d_dbias != nullptr;
            q.sums[0] = a->d_dbias;
            q.sums_dtype = a->wgrad_dtype;
            q.partial = (float *)a->d_ws;
            ECF_TRY(launch_dense_grad(q, &sums, st));
            gx.unscale = q.row_inverse, gw.unscale = q.col_inverse;
            gx.a[0] = q.dz, gw.a[0] = q.scaled ? q.dz_w : q.dz;
        }
        if (direct)
            gx.a[0] = gw.a[0] = a->d_dout;
        const int64_t lddz = direct ? lddy : w.pitch;
        gx.dtype = gx.out_dtype = gw.dtype = a->dtype;
        gx.b_t = gw.a_t = gw.b_t = true;
        gx.ksegs = gx.mhalves = gw.ksegs = gw.mhalves = 1;
        gx.lda = gw.lda = lddz;
        gx.a_padded = gw.a_padded = !direct;
        gx.b[0] = a->d_w;
        gx.ldb = ldw;
        gx.M = T, gx.N = a->in_features, gx.K = a->out_features;
        gx.out[0] = a->d_dx;
        gx.ldout = lddx;
        gw.out_dtype = a->wgrad_dtype;
        gw.b[0] = a->d_x;
        gw.ldb = ldx;
        gw.M = a->out_features, gw.N = a->in_features, gw.K = T;
        gw.out[0] = a->d_dw;
        gw.ldout = lddw;
        return launch_dense_backward(want_dx ? &gx : nullptr, a->d_dw ? &gw : nullptr, sums, (char *)a->d_ws + w.split,
                                     w.room, st);
    });
}

}  // extern "C"
