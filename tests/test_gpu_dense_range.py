"""GPU tests of the dense operators' range: gradients whose da, db or dz lie outside
fp16's range although their products do not, and infinities that meet in fp32."""
import pytest
import torch

import dense_ref as R
from expert_cache_ffn_amd.layer import GatedProjection, Linear
from gpu_util import say

pytestmark = pytest.mark.gpu

F16 = torch.float16


def rand(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def scaled_half(*ds):
    """Bounds of the [(value, bound unrounded, ...)] of R.grads once held in fp16 times the power of two that
    puts the largest of them all at 2^14 to 2^15: half a step of each value, and half a subnormal step
    (2^-25) on that scale, 2^-39 of the largest."""
    top = max(float(d[d.isfinite()].abs().max()) for d, _, _ in ds)
    return [(d, e, e + d.abs() * (2.0 ** -11 * (1 + 1e-3)) + top * 2.0 ** -39) for d, e, _ in ds]


# kernels of few and many tokens, aligned and odd widths, rows under 8 elements, split and unsplit products
SHAPES = [(64, 256, 128), (1, 40, 72), (5, 7, 3), (300, 512, 136), (777, 133, 201), (2049, 264, 513), (40, 4096, 1024),
          (4100, 64, 1100)]  # (the last: more tiles than blocks that look for the largest)


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dy,ws", [(1e-9, 1e3), (3e8, 1e-6), (1e-5, 1.0)])
@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_fp16_linear_gradients_from_an_fp32_stream(act, dy, ws, T, K, N):
    say(f"case: fp16 range, linear {act} dy {dy} w {ws} T {T} K {K} N {N}")
    x, w = rand(1, T, K, dtype=F16), rand(2, N, K, std=ws, dtype=F16)
    z, dout = rand(6, T, N, dtype=F16), rand(8, T, N, std=dy)
    dx, dw, db = Linear(w, rand(4, N, dtype=F16), act=act, out_dtype=torch.float32).backward(
        x, dout, z=z, w_grad_dtype=torch.float32)
    (dz, e, r), = scaled_half(*R.grads(dout.double(), z.double(), act, F16))
    R.check("dx", dx, R.rounded(*R.product(dz, w.double().t().contiguous(), r), F16))
    R.check("dw", dw, R.rounded(*R.product(dz.t(), x.double().t(), r.t()), torch.float32))
    R.check("dbias", db, R.colsum(dz, e, torch.float32))


@pytest.mark.parametrize("T,d,I", SHAPES)
@pytest.mark.parametrize("std_h,std_b,std_w", [(30.0, 1e4, 1e-6), (1e-4, 1e-4, 1e3), (0.02, 1.0, 0.05)])
def test_fp16_gated_gradients_out_of_range(std_h, std_b, std_w, T, d, I):
    say(f"case: fp16 range, gated dh {std_h} b {std_b} w {std_w} T {T} d {d} I {I}")
    x, wg, wu = rand(1, T, d, dtype=F16), rand(2, I, d, std=std_w, dtype=F16), rand(3, I, d, std=std_w, dtype=F16)
    a, b, dh = rand(6, T, I, dtype=F16), rand(7, T, I, std=std_b, dtype=F16), rand(8, T, I, std=std_h, dtype=F16)
    a, b, dh = a.clamp(-9, 9), b.clamp(-6e4, 6e4), dh.clamp(-200, 200)
    outs = GatedProjection(wg, wu).backward(x, a, b, dh, w_grad_dtype=torch.float32)
    (da, _, ra), (db, _, rb) = scaled_half(*R.grads(dh.double(), a.double(), "silu", F16, b.double()))
    both = torch.cat([wg, wu], 0).double().t().contiguous()
    R.check("dx", outs[0], R.rounded(*R.product(torch.cat([da, db], 1), both, torch.cat([ra, rb], 1)), F16))
    R.check("dw_gate", outs[1], R.rounded(*R.product(da.t(), x.double().t(), ra.t()), torch.float32))
    R.check("dw_up", outs[2], R.rounded(*R.product(db.t(), x.double().t(), rb.t()), torch.float32))


@pytest.mark.parametrize("scale", [2.0 ** 125, 1e30, 1.0, 1e-30, 2.0 ** -126, 2.0 ** -140])
def test_fp16_weight_gradients_over_the_fp32_exponents(scale):
    """dW in fp32 from an fp32 dy of any size.  (From 2^-112 down the power of two stays at 2^126: half a
    subnormal step is 2^-151.)"""
    say(f"case: fp16 range, dy {scale}")
    T, K, N = 70, 96, 40
    x, w, dout = rand(1, T, K, dtype=F16), rand(2, N, K, dtype=F16), (rand(8, T, N).clamp(-3.9, 3.9).double() * scale).float()
    dw = Linear(w, out_dtype=torch.float32).backward(x, dout, w_grad_dtype=torch.float32, need_dx=False)[1]
    (dz, e, r), = scaled_half(*R.grads(dout.double(), dout.double(), "none", F16))
    ref, err = R.product(dz.t(), x.double().t(), (r + 2.0 ** -151).t())
    ref, err = R.rounded(ref, err, torch.float32)
    # (sums of 70 products of up to 2^127 x 4 pass fp32's largest value: those round to infinity)
    fits, past = (ref.abs() + err < torch.finfo(torch.float32).max), (ref.abs() - err > torch.finfo(torch.float32).max)
    R.check("dw", dw[fits], (ref[fits], err[fits]))
    assert torch.equal(dw[past].double(), torch.sign(ref[past]) * float("inf"))


@pytest.mark.parametrize("T", [3, 70, 600])
def test_fp16_scale_and_special_values(T):
    """The scale is that of the finite gradients: infinities and NaN change only what they are part of, and
    no gradient at all is a gradient of zeros."""
    say(f"case: fp16 range, special values T {T}")
    K, N = 136, 72
    x, w, dout = rand(1, T, K, dtype=F16), rand(2, N, K, std=1e3, dtype=F16), rand(8, T, N, std=1e-8)
    lin = Linear(w, out_dtype=torch.float32)
    (dz, e, r), = scaled_half(*R.grads(dout.double(), dout.double(), "none", F16))
    refx = R.rounded(*R.product(dz, w.double().t().contiguous(), r), F16)
    refw = R.rounded(*R.product(dz.t(), x.double().t(), r.t()), torch.float32)
    rows, cols = torch.arange(T, device="cuda") != T // 2, torch.arange(N, device="cuda") != 9
    for bad in (float("inf"), float("-inf"), float("nan")):
        db = dout.clone()
        db[T // 2, 9] = bad
        dx, dw, _ = lin.backward(x, db, w_grad_dtype=torch.float32)
        R.check("dx", dx[rows], [v[rows] for v in refx])
        R.check("dw", dw[cols], [v[cols] for v in refw])
        assert not dx[T // 2].isfinite().any() and not dw[9].isfinite().any()
    dx, dw, _ = lin.backward(x, torch.zeros_like(dout), w_grad_dtype=torch.float32)
    assert not dx.any() and not dw.any()
    dx, dw, _ = lin.backward(x, torch.full_like(dout, float("inf")), w_grad_dtype=torch.float32)
    assert not dx.isfinite().any() and not dw.isfinite().any()


def test_fp16_range_in_a_captured_graph():
    """Each replay finds the scale of its own gradients."""
    T, K, N = 200, 136, 264
    x, w = rand(1, T, K, dtype=F16), rand(2, N, K, dtype=F16)
    lin = Linear(w, out_dtype=torch.float32)
    douts = [rand(8 + i, T, N, std=s) for i, s in enumerate((1e-9, 1e7, 1.0, 1e-20))]
    want = [lin.backward(x, t, w_grad_dtype=torch.float32) for t in douts]
    torch.cuda.synchronize()
    cur, side, g = douts[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        outs = lin.backward(x, cur, w_grad_dtype=torch.float32)
    for i in (1, 0, 2, 3, 1, 2):
        cur.copy_(douts[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(p is None or torch.equal(p, q) for p, q in zip(outs, want[i])), f"replay of gradients {i} differs"
        again = lin.backward(x, douts[(i + 1) % 4], w_grad_dtype=torch.float32)
        assert all(p is None or torch.equal(p, q) for p, q in zip(again, want[(i + 1) % 4]))


def kind(t):
    """0 finite, 1 NaN, 2 infinity, -2 minus infinity."""
    t = t.double().cpu()
    return torch.where(t.isnan(), 1, torch.where(t.isinf(), 2 * torch.sign(t), 0.0))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,N", [(5, 40, 24), (64, 200, 150), (65, 200, 150), (300, 137, 131), (1000, 264, 520), (70, 6, 5)])
def test_infinities_and_nans_that_meet(T, K, N, dt):
    """Infinities of either sign against infinities, zeros, NaN and finite values at the same k: every kernel
    gives what IEEE products and sums give, whatever the sizes."""
    say(f"case: infinities that meet T {T} K {K} N {N} {dt}")
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": F16}[dt]
    inf, nan = float("inf"), float("nan")
    x, w = rand(1, T, K, dtype=dtype), rand(2, N, K, dtype=dtype)
    for i, v in enumerate((inf, -inf, inf, nan, 0.0)):  # rows of x and of w that hold one each, all at k 3
        x[(7 * i + 1) % T, 3] = v
        w[(3 * i + 2) % N, 3] = v
    x[T - 1, K - 1], w[N - 1, K - 1] = -inf, inf
    x[0, 0] = inf
    w[0, 0], w[1, 0] = 0.0, -inf
    ref = kind(x.double().cpu() @ w.double().cpu().t())
    assert {-2.0, 1.0, 2.0} <= set(ref.unique().tolist())
    assert torch.equal(kind(Linear(w, out_dtype=torch.float32).forward(x)), ref)
    _, a, b = GatedProjection(w, w, act="none").forward(x, save=True)
    assert torch.equal(kind(a), ref) and torch.equal(kind(b), ref)
    # the same product as dz W and as dz^T x (without an activation dy is dz)
    wt = w.t().contiguous()
    assert torch.equal(kind(Linear(wt).backward(rand(3, T, N, dtype=dtype), x, need_dw=False)[0]), ref)
    dw = Linear(rand(4, T, N, dtype=dtype)).backward(wt, x.t().contiguous(), need_dx=False)[1]
    assert torch.equal(kind(dw), ref)


@pytest.mark.parametrize("T,d,I", [(6, 40, 72), (70, 256, 128), (333, 133, 201), (700, 512, 1000)])
@pytest.mark.parametrize("huge", [6e4, 1e3, 0.0])
def test_fp16_rows_and_columns_keep_apart(huge, T, d, I):
    """Rows of huge gradients (padding, say) leave the other rows' dx as it is without them, to the bit, and
    columns of huge gradients the other rows of dW."""
    say(f"case: fp16 range, huge {huge} rows and columns T {T} d {d} I {I}")
    x, wg, wu = rand(1, T, d, dtype=F16), rand(2, I, d, std=.05, dtype=F16), rand(3, I, d, std=.05, dtype=F16)
    a, b, dh = rand(6, T, I, dtype=F16), rand(7, T, I, dtype=F16), rand(8, T, I, std=1e-4, dtype=F16)
    gp, rows, cols = GatedProjection(wg, wu), torch.arange(T, device="cuda") % 3 != 1, torch.arange(I, device="cuda") % 5 != 2
    dx, dwg, dwu, *_ = gp.backward(x, a, b, dh, w_grad_dtype=torch.float32)
    for t in (a, b, dh):
        t[~rows] = huge
    assert torch.equal(gp.backward(x, a, b, dh)[0][rows], dx[rows])
    a, b, dh = rand(6, T, I, dtype=F16), rand(7, T, I, dtype=F16), rand(8, T, I, std=1e-4, dtype=F16)
    for t in (a, b, dh):
        t[:, ~cols] = huge
    outs = gp.backward(x, a, b, dh, w_grad_dtype=torch.float32)
    assert torch.equal(outs[1][cols], dwg[cols]) and torch.equal(outs[2][cols], dwu[cols])
    lin = Linear(wg, out_dtype=torch.float32)
    dy = rand(9, T, I, std=1e-6)
    dx, dw, _ = lin.backward(x, dy, w_grad_dtype=torch.float32)
    far = dy.clone()
    far[~rows] = huge * 1e20
    assert torch.equal(lin.backward(x, far)[0][rows], dx[rows])
    far = dy.clone()
    far[:, ~cols] = huge * 1e20
    assert torch.equal(lin.backward(x, far, w_grad_dtype=torch.float32)[1][cols], dw[cols])


def own_scales(*ds):
    """As scaled_half, of the scales of rows (for dx) and of columns (for dW): [(value, bound for dx, for dW)]."""
    fin = [torch.where(d.isfinite(), d.abs(), 0.0) for d, _, _ in ds]
    row = torch.cat(fin, 1).amax(1, keepdim=True)
    return [(d, e + d.abs() * (2.0 ** -11 * (1 + 1e-3)) + row * 2.0 ** -39,
             e + d.abs() * (2.0 ** -11 * (1 + 1e-3)) + f.amax(0, keepdim=True) * 2.0 ** -39) for (d, e, _), f in zip(ds, fin)]


@pytest.mark.parametrize("T,d,I", SHAPES)
def test_fp16_gradients_of_rows_and_columns_of_every_size(T, d, I):
    """dz from 1e-30 to 1e30 within one call: each row of dx and of dW is as near as if it were alone."""
    say(f"case: fp16 range, every size T {T} d {d} I {I}")
    x, w = rand(1, T, d, dtype=F16), rand(2, I, d, dtype=F16)
    lin = Linear(w, rand(4, I, dtype=F16), act="silu", out_dtype=torch.float32)
    z = rand(6, T, I, dtype=F16)
    size_t, size_n = torch.logspace(-30, 4, T, device="cuda")[:, None], torch.logspace(-30, 30, I, device="cuda")[None]
    dy = rand(8, T, I) * size_t
    dx = lin.backward(x, dy, z)[0]
    (dz, r, _), = own_scales(*R.grads(dy.double(), z.double(), "silu", F16))
    ref, err = R.rounded(*R.product(dz, w.double().t().contiguous(), r), F16)
    fits = ref.abs() + err < 65504
    R.check("dx", dx[fits], (ref[fits], err[fits]))
    dy = rand(8, T, I) * size_n
    dw = lin.backward(x, dy, z, w_grad_dtype=torch.float32)[1]
    (dz, _, r), = own_scales(*R.grads(dy.double(), z.double(), "silu", F16))
    R.check("dw", dw, R.rounded(*R.product(dz.t(), x.double().t(), r.t()), torch.float32))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_fp16_slopes_above_one(act, T, K, N):
    """A linear dz of an fp16 dy near the type's largest value: slopes of up to 1.13 carry it past 65504."""
    say(f"case: fp16 range, {act} slopes T {T} K {K} N {N}")
    x, w = rand(1, T, K, dtype=F16), rand(2, N, K, std=1e-3, dtype=F16)
    z = (rand(6, T, N).double().clamp(-1, 1) * .3 + 1.5).half()
    dout = (torch.sign(rand(8, T, N)) * (65504 - 2000 * rand(9, T, N).abs())).half()
    assert float((dout.double() * R.act_both(z.double(), act)[1]).abs().max()) > 65520
    dx, dw, db = Linear(w, rand(4, N, dtype=F16), act=act).backward(x, dout, z, w_grad_dtype=torch.float32)
    (dz, e, _), = R.grads(dout.double(), z.double(), act, F16)
    (_, rx, rw), = own_scales((dz, e, None))
    ref, err = R.rounded(*R.product(dz, w.double().t().contiguous(), rx), F16)
    fits = ref.abs() + err < 65504
    R.check("dx", dx[fits], (ref[fits], err[fits]))
    R.check("dw", dw, R.rounded(*R.product(dz.t(), x.double().t(), rw.t()), torch.float32))
    R.check("dbias", db, R.colsum(dz, e, torch.float32))


def product_of_subnormals(a, b, da):
    """R.product where operands are subnormal in fp16.  The matrix instruction aligns its 16 products by the
    exponents of their operands, in which a subnormal counts as 2^-14, before it adds them in fp32: beside
    1 * 2^-18, whose exponents say 2^-14, a product of 2^-40 is 2^-26 of that and is lost whole (measured).  So
    the rounding of an addition, 2^-23 of the sum so far, is one of products whose operands are at least 2^-14."""
    z, err = R.product(a, b, da)
    low = 2.0 ** -14
    return z, err + (a.abs().clamp_min(low) @ b.abs().clamp_min(low).t()) * ((a.shape[1] + 2) * R.EPS23)


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_fp16_linear_gradients_of_small_fp16_dy(T, K, N):
    """dy of 2^-20 and less, all subnormal: dz keeps its bits."""
    say(f"case: fp16 range, small fp16 dy T {T} K {K} N {N}")
    x, w = rand(1, T, K, dtype=F16), rand(2, N, K, std=1e2, dtype=F16)
    z, dout = rand(6, T, N, dtype=F16), rand(8, T, N, std=1e-6, dtype=F16)
    for act in ("gelu", "relu"):
        dx, dw, _ = Linear(w, act=act).backward(x, dout, z, w_grad_dtype=torch.float32)
        (dz, e, _), = R.grads(dout.double(), z.double(), act, F16)
        (_, rx, rw), = own_scales((dz, e, None)) if act == "gelu" else [(dz, e, e)]  # (relu's dz is exact)
        product = R.product if act == "gelu" else product_of_subnormals
        R.check("dx", dx, R.rounded(*product(dz, w.double().t().contiguous(), rx), F16))
        R.check("dw", dw, R.rounded(*product(dz.t(), x.double().t(), rw.t()), torch.float32))
