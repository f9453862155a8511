// C-ABI entry points of the low-rank adapters: argument checks, workspaces, and the
// kernels each call is made of.
#include <algorithm>
#include <cstdint>

#include "tokens_internal.h"

namespace ecf {
namespace {

constexpr int32_t kMaxAdapters = 1024, kMaxRank = 256;

int check_shape(const char *what, int32_t K, int32_t N, int32_t r, int32_t n, int32_t T)
{
    if (K < 1 || K > kTokenMax || N < 1 || N > kTokenMax || T < 0 || T > kTokenMax)
        return set_error(ECF_EINVAL, "%s: widths must be 1..%d and n_tokens 0..%d (in=%d, out=%d, T=%d)", what, kTokenMax,
                         kTokenMax, K, N, T);
    if (r < 1 || r > kMaxRank || n < 1 || n > kMaxAdapters)
        return set_error(ECF_EINVAL, "%s: rank must be 1..%d and n_adapters 1..%d (rank=%d, n_adapters=%d)", what, kMaxRank,
                         kMaxAdapters, r, n);
    return ECF_OK;
}

// The order where the caller gives none, the splits' parts of h, and in the backward pass
// g and the outer products' slots.
struct Workspace {
    size_t counts, offsets, tiles, order, place, sort, sort_bytes, part, g, slots_a, slots_b, total;
    int splits;
};
Workspace workspace(int32_t K, int32_t N, int32_t r, int32_t n, int32_t T, bool backward)
{
    Workspace w{};
    auto take = [&](size_t bytes) {
        const size_t at = w.total;
        w.total += al256(bytes);
        return at;
    };
    const int32_t reduced = backward ? N : K;
    const bool few = !backward && T <= kAdapterFew;
    w.splits = few ? 1 : shrink_splits(T, reduced);
    if (!few) {
        w.counts = take((size_t)n * 4);
        w.offsets = take((size_t)(n + 1) * 4);
        w.tiles = take((size_t)(n + 2) * 4);
        w.order = take((size_t)T * 4);
        w.place = take((size_t)T * 4);
        w.sort_bytes = sort_ws(T, n);
        w.sort = take(w.sort_bytes);
    }
    // (a size query does not know the type: what holds for the widest holds for all)
    if (!few || !adapter_few_in_one(T, K, N, r, 4))
        w.part = take((size_t)shrink_rows(T) * r * 4);
    if (backward) {
        w.g = take((size_t)T * r * 4);
        w.slots_a = take(outer_slots(outer_chunks(T, outer_slices(K)), K, r));
        w.slots_b = take(outer_slots(outer_chunks(T, outer_slices(N)), N, r));
    }
    return w;
}

int check_args(const char *what, const ecf_adapter_args *a, int32_t T)
{
    if (!a)
        return set_error(ECF_EINVAL, "%s: args is NULL", what);
    ECF_TRY(check_shape(what, a->in_features, a->out_features, a->rank, a->n_adapters, T));
    if (!dense_dtype(a->dtype))
        return set_error(ECF_EINVAL, "%s: dtype must be ECF_F32, ECF_BF16 or ECF_F16 (got %d)", what, a->dtype);
    if (a->out_dtype != a->dtype && a->out_dtype != ECF_F32)
        return set_error(ECF_EINVAL, "%s: out_dtype must be dtype or ECF_F32 (got %d)", what, a->out_dtype);
    if (a->idx_bytes != 4 && a->idx_bytes != 8)
        return set_error(ECF_EINVAL, "%s: idx_bytes must be 4 or 8 (got %d)", what, a->idx_bytes);
    if (!a->d_order != !a->d_offsets || !a->d_order != !a->d_tiles)
        return set_error(ECF_EINVAL, "%s: d_order, d_offsets and d_tiles come together", what);
    ECF_TRY(check_aligned(what, "d_order", a->d_order, 4));
    ECF_TRY(check_aligned(what, "d_offsets", a->d_offsets, 4));
    ECF_TRY(check_aligned(what, "d_tiles", a->d_tiles, 4));
    ECF_TRY(check_aligned(what, "d_scale", a->d_scale, 4));
    return check_aligned(what, "d_h", a->d_h, 4);
}

// The tokens' order: the caller's, or one made in the workspace.
int make_order(const ecf_adapter_args *a, int32_t T, const Workspace &w, AdapterOrder *o)
{
    *o = {a->d_idx, a->idx_bytes == 8, a->d_order, a->d_offsets, a->d_tiles, T, a->n_adapters};
    if (a->d_order)
        return ECF_OK;
    char *ws = (char *)a->d_ws;
    SortCall s{};
    s.T = T, s.k = 1, s.E = a->n_adapters, s.wide = o->wide;
    s.idx = a->d_idx, s.ldidx = 1;
    s.counts = (int32_t *)(ws + w.counts), s.offsets = (int32_t *)(ws + w.offsets), s.tiles = (int32_t *)(ws + w.tiles);
    s.order = (int32_t *)(ws + w.order), s.place = (int32_t *)(ws + w.place);
    s.segments = (int32_t *)(ws + w.sort);
    ECF_TRY(launch_token_sort(s, (hipStream_t)a->stream));
    o->order = s.order, o->offsets = s.offsets, o->tiles = s.tiles;
    return ECF_OK;
}

}  // namespace

// K per split: up to four blocks a CU where there are few tiles, at most 7 splits (each adds a part
// of h that every block of the expand reads) and one for each 256 of K, in whole chunks.
int shrink_split_k(int T, int K)
{
    int s = kShrinkBlocks / (T / kTileRows + 1);
    s = s < kShrinkSplits ? s : kShrinkSplits;
    const int most = (K + 255) / 256;
    s = s < most ? s : most;
    s = s > 1 ? s : 1;
    return ((K + s - 1) / s + kShrinkChunk - 1) / kShrinkChunk * kShrinkChunk;
}

// Splits that have any of K.
int shrink_splits(int T, int K)
{
    const int k = shrink_split_k(T, K);
    return (K + k - 1) / k;
}

int outer_slices(int W) { return (W + kOuterCols - 1) / kOuterCols; }

// Runs of the sorted rows: two blocks a CU over all slices, 128 rows each at least.
int outer_chunks(int T, int slices)
{
    const int most = (T + 127) / 128, s = 512 / slices;
    return s < 1 || most < 1 ? 1 : s < most ? s : most;
}

}  // namespace ecf

using namespace ecf;

extern "C" {

size_t ecf_adapter_workspace_bytes(int32_t in_features, int32_t out_features, int32_t rank, int32_t n_adapters,
                                   int32_t n_tokens, int32_t backward)
{
    if (check_shape("ecf_adapter_workspace_bytes", in_features, out_features, rank, n_adapters, n_tokens) != ECF_OK)
        return SIZE_MAX;
    return workspace(in_features, out_features, rank, n_adapters, n_tokens, backward != 0).total;
}

int ecf_adapter_forward(const ecf_adapter_args *a, int32_t T)
{
    return guarded("ecf_adapter_forward", [&]() -> int {
        const char *me = "ecf_adapter_forward";
        ECF_TRY(check_args(me, a, T));
        if (T == 0)
            return ECF_OK;
        const int64_t K = a->in_features, N = a->out_features;
        const int64_t ldx = ld_or(a->ld_x, K), ldres = ld_or(a->ld_residual, N), ldout = ld_or(a->ld_out, N);
        ECF_TRY(check_present(me, "d_idx", a->d_idx, (size_t)a->idx_bytes));
        ECF_TRY(check_rows(me, "d_x", a->d_x, ldx, K, a->dtype));
        ECF_TRY(check_rows(me, "d_a", a->d_a, K, K, a->dtype));
        ECF_TRY(check_rows(me, "d_b", a->d_b, a->rank, a->rank, a->dtype));
        ECF_TRY(check_rows(me, "d_out", a->d_out, ldout, N, a->out_dtype));
        if (a->d_residual)
            ECF_TRY(check_rows(me, "d_residual", a->d_residual, ldres, N, a->out_dtype));
        const Workspace w = workspace(a->in_features, a->out_features, a->rank, a->n_adapters, T, false);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, w.total));
        ECF_TRY(check_apart(me, {{"d_out", a->d_out}, {"d_h", a->d_h}, {"d_ws", w.total ? a->d_ws : nullptr}},
                            {{"d_x", a->d_x}, {"d_a", a->d_a}, {"d_b", a->d_b}, {"d_scale", a->d_scale}, {"d_idx", a->d_idx},
                             {"d_order", a->d_order}, {"d_offsets", a->d_offsets}, {"d_tiles", a->d_tiles}}));
        ECF_TRY(check_apart(me, {{"d_h", a->d_h}, {"d_ws", w.total ? a->d_ws : nullptr}}, {{"d_residual", a->d_residual}}));
        ECF_TRY(check_same_stride(me, "d_out", a->d_out, ldout, "d_residual", a->d_residual, ldres));
        hipStream_t st = (hipStream_t)a->stream;
        const bool few = T <= kAdapterFew;
        ShrinkCall s{};
        ExpandCall e{};
        if (few)
            s.o = {a->d_idx, a->idx_bytes == 8, nullptr, nullptr, nullptr, T, a->n_adapters};
        else
            ECF_TRY(make_order(a, T, w, &s.o));
        e.o = s.o;
        s.dtype = s.x_dtype = a->dtype;
        s.K = a->in_features, s.r = a->rank;
        s.m = a->d_a, s.x = a->d_x, s.ldx = ldx;
        s.part = (float *)((char *)a->d_ws + w.part);
        s.splits = w.splits, s.split_k = shrink_split_k(T, s.K);
        e.dtype = a->dtype, e.out_dtype = a->out_dtype;
        e.N = a->out_features, e.r = a->rank;
        e.m = a->d_b, e.scale = a->d_scale;
        e.part = s.part, e.splits = w.splits;
        e.h = a->d_h;
        e.residual = a->d_residual, e.ldres = ldres;
        e.out = a->d_out, e.ldout = ldout;
        if (few && adapter_few_in_one(T, K, N, a->rank, 4))
            return launch_few(s, e, st);
        ECF_TRY(few ? launch_few_shrink(s, st) : launch_shrink(s, st));
        return few ? launch_few_expand(e, st) : launch_expand(e, st);
    });
}

int ecf_adapter_backward(const ecf_adapter_args *a, int32_t T)
{
    return guarded("ecf_adapter_backward", [&]() -> int {
        const char *me = "ecf_adapter_backward";
        ECF_TRY(check_args(me, a, T));
        ECF_TRY(check_grad_dtype(me, a->wgrad_dtype, a->dtype));
        const int64_t K = a->in_features, N = a->out_features;
        const int64_t ldx = ld_or(a->ld_x, K), ldres = ld_or(a->ld_residual, K), lddy = ld_or(a->ld_dout, N),
                      lddx = ld_or(a->ld_dx, K);
        const bool want_dx = a->d_dx && T > 0;
        if (T > 0) {
            ECF_TRY(check_present(me, "d_idx", a->d_idx, (size_t)a->idx_bytes));
            ECF_TRY(check_rows(me, "d_dout", a->d_dout, lddy, N, a->out_dtype));
            if (want_dx || a->d_da)
                ECF_TRY(check_rows(me, "d_b", a->d_b, a->rank, a->rank, a->dtype));
            if (a->d_da)
                ECF_TRY(check_rows(me, "d_x", a->d_x, ldx, K, a->dtype));
            if (a->d_db)
                ECF_TRY(check_present(me, "d_h", a->d_h, 4));
        }
        if (want_dx) {
            ECF_TRY(check_rows(me, "d_a", a->d_a, K, K, a->dtype));
            ECF_TRY(check_rows(me, "d_dx", a->d_dx, lddx, K, a->dtype));
            if (a->d_residual)
                ECF_TRY(check_rows(me, "d_residual", a->d_residual, ldres, K, a->dtype));
        }
        ECF_TRY(check_vector(me, "d_da", a->d_da, a->wgrad_dtype));
        ECF_TRY(check_vector(me, "d_db", a->d_db, a->wgrad_dtype));
        const Workspace w = workspace(a->in_features, a->out_features, a->rank, a->n_adapters, T, true);
        ECF_TRY(check_ws(me, a->d_ws, a->ws_bytes, w.total));
        ECF_TRY(check_apart(me, {{"d_dx", a->d_dx}, {"d_da", a->d_da}, {"d_db", a->d_db}, {"d_ws", a->d_ws}},
                            {{"d_x", a->d_x}, {"d_a", a->d_a}, {"d_b", a->d_b}, {"d_scale", a->d_scale}, {"d_idx", a->d_idx},
                             {"d_order", a->d_order}, {"d_offsets", a->d_offsets}, {"d_tiles", a->d_tiles}, {"d_h", a->d_h},
                             {"d_dout", a->d_dout}}));
        ECF_TRY(check_apart(me, {{"d_da", a->d_da}, {"d_db", a->d_db}, {"d_ws", a->d_ws}}, {{"d_residual", a->d_residual}}));
        ECF_TRY(check_same_stride(me, "d_dx", a->d_dx, lddx, "d_residual", a->d_residual, ldres));
        if (!want_dx && !a->d_da && !a->d_db)
            return ECF_OK;
        hipStream_t st = (hipStream_t)a->stream;
        char *ws = (char *)a->d_ws;
        AdapterOrder o{};
        ECF_TRY(make_order(a, T, w, &o));
        float *g = (float *)(ws + w.g);
        if (T > 0 && (want_dx || a->d_da)) {
            ShrinkCall s{};
            s.o = o;
            s.dtype = a->dtype, s.x_dtype = a->out_dtype;
            s.K = a->out_features, s.r = a->rank;
            s.of_b = true;
            s.m = a->d_b, s.x = a->d_dout, s.ldx = lddy;
            s.part = (float *)(ws + w.part);
            s.splits = w.splits, s.split_k = shrink_split_k(T, s.K);
            ECF_TRY(launch_shrink(s, st));
            ExpandCall e{};
            e.o = o;
            e.dtype = e.out_dtype = a->dtype;
            e.N = a->in_features, e.r = a->rank;
            e.of_a = true;
            e.m = a->d_a, e.scale = a->d_scale;
            e.part = s.part, e.splits = w.splits;
            e.h = a->d_da ? g : nullptr;
            e.scaled = true;
            e.residual = a->d_residual, e.ldres = ldres;
            e.out = want_dx ? a->d_dx : nullptr, e.ldout = lddx;
            ECF_TRY(launch_expand(e, st));
        }
        // both in one launch where x and dout are of one type (more slices, so no more runs
        // than either has room for)
        OuterCall q[2]{};
        int n = 0;
        for (int of_b = 0; of_b < 2; ++of_b) {
            void *d = of_b ? a->d_db : a->d_da;
            if (!d)
                continue;
            OuterCall &c = q[n++];
            c.o = o;
            c.x_dtype = of_b ? a->out_dtype : a->dtype, c.grad_dtype = a->wgrad_dtype;
            c.W = of_b ? a->out_features : a->in_features, c.r = a->rank;
            c.of_b = of_b;
            c.g = of_b ? a->d_h : g, c.gscale = of_b ? a->d_scale : nullptr;
            c.x = of_b ? a->d_dout : a->d_x, c.ldx = of_b ? lddy : ldx;
            c.d = d;
            c.slots = (float *)(ws + (of_b ? w.slots_b : w.slots_a));
        }
        if (n == 2 && q[0].x_dtype == q[1].x_dtype)
            return launch_outer(q, 2, outer_chunks(T, outer_slices(q[0].W) + outer_slices(q[1].W)), st);
        for (int i = 0; i < n; ++i)
            ECF_TRY(launch_outer(q + i, 1, outer_chunks(T, outer_slices(q[i].W)), st));
        return ECF_OK;
    });
}

}  // extern "C"
