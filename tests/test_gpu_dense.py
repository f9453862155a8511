"""GPU tests of the dense feed-forward operators against the 64-bit reference of
dense_ref.py: types, activations, odd sizes, strides and alignment, long
offsets, special values, streams, graphs, and the block they form together."""
import numpy as np
import pytest
import torch

import dense_ref as R
import ecf_synth as syn
import expert_cache_ffn_amd as ecf
from expert_cache_ffn_amd.layer import GatedProjection, Linear
from gpu_util import Case, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "none"]


def rand(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def strided(t, pad, shift):
    """The same values in rows `pad` elements further apart, starting `shift` elements in; the
    gaps hold NaN.  Returns (view, whole buffer)."""
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((rows * ld + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v, buf


def d64(*ts):
    return [None if t is None else t.double() for t in ts]


# (tokens, d, I): one of everything, single rows and columns, sizes off every tile and vector width, and
# sizes where each kind of call changes its tiles
SIZES = [(1, 1, 1), (1, 8, 3), (2, 7, 1), (3, 65, 17), (4, 64, 64), (5, 130, 36), (8, 520, 100), (16, 256, 128),
         (17, 1000, 33), (31, 96, 264), (33, 72, 200), (64, 256, 128), (65, 129, 131), (100, 512, 72), (127, 257, 255),
         (128, 128, 128), (200, 264, 520), (257, 320, 65), (300, 136, 1030), (513, 200, 392)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,I", SIZES)
def test_gated_forward(T, d, I, dt):
    say(f"case: gated forward T {T} d {d} I {I} {dt}")
    dtype = DT[dt]
    x, wg, wu = rand(1, T, d, dtype=dtype), rand(2, I, d, std=d ** -.5, dtype=dtype), rand(3, I, d, std=d ** -.5, dtype=dtype)
    act = ACTS[(T + d + I) % 4]
    bg, bu = (rand(4, I, dtype=dtype), rand(5, I, dtype=dtype)) if (d + I) % 2 else (None, None)
    layer = GatedProjection(wg, wu, bg, bu, act=act)
    ref = R.gated_forward(*d64(x, wg, wu, bg, bu), act, dtype)
    h, a, b = layer.forward(x, save=True)
    for name, got in (("h", h), ("a", a), ("b", b)):
        R.check(name, got, ref[name])
    assert torch.equal(layer.forward(x), h), "saving changes h, or two calls differ"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,I", SIZES)
def test_gated_backward(T, d, I, dt):
    say(f"case: gated backward T {T} d {d} I {I} {dt}")
    dtype = DT[dt]
    x, wg, wu = rand(1, T, d, dtype=dtype), rand(2, I, d, std=d ** -.5, dtype=dtype), rand(3, I, d, std=d ** -.5, dtype=dtype)
    a, b, dh = rand(6, T, I, dtype=dtype), rand(7, T, I, dtype=dtype), rand(8, T, I, std=0.1, dtype=dtype)
    act = ACTS[(T + d + I) % 5]
    gd = torch.float32 if T % 2 else dtype
    bg = rand(4, I, dtype=dtype) if I % 3 else None
    bu = rand(5, I, dtype=dtype) if I % 2 else None
    layer = GatedProjection(wg, wu, bg, bu, act=act)
    ref = R.gated_backward(*d64(x, wg, wu, a, b, dh), act, dtype, gd)
    outs = layer.backward(x, a, b, dh, w_grad_dtype=gd)
    for name, got in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), outs):
        if name == "db_gate" and bg is None or name == "db_up" and bu is None:
            assert got is None
        else:
            R.check(name, got, ref[name])
    again = layer.backward(x, a, b, dh, w_grad_dtype=gd)
    assert all(p is None or torch.equal(p, q) for p, q in zip(outs, again)), "two calls differ"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_forward(T, K, N, dt):
    say(f"case: linear forward T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    out_dtype = torch.float32 if (T + N) % 2 else dtype
    x, w = rand(1, T, K, dtype=dtype), rand(2, N, K, std=K ** -.5, dtype=dtype)
    bias = rand(4, N, dtype=dtype) if K % 2 == 0 else None
    residual = rand(5, T, N, dtype=out_dtype) if T % 3 else None
    act = ACTS[(T + K + N) % 5]
    layer = Linear(w, bias, act=act, out_dtype=out_dtype)
    ref = R.linear_forward(*d64(x, w, bias), act, None if residual is None else residual.double(), dtype, out_dtype)
    y, z = layer.forward(x, residual=residual, save=True)
    R.check("z", z, ref["z"])
    R.check("y", y, ref["y"])
    if residual is not None:  # into the residual itself
        run = residual.clone()
        assert layer.forward(x, residual=run, out=run) is run
        assert torch.equal(run, y), "in place differs"
    else:
        assert torch.equal(layer.forward(x), y)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_backward(T, K, N, dt):
    say(f"case: linear backward T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    out_dtype = torch.float32 if (T + N) % 2 else dtype
    gd = torch.float32 if K % 2 else dtype
    act = ACTS[(T + K + N) % 5]
    x, w = rand(1, T, K, dtype=dtype), rand(2, N, K, std=K ** -.5, dtype=dtype)
    z, dout = rand(6, T, N, dtype=dtype), rand(8, T, N, std=0.1, dtype=out_dtype)
    bias = rand(4, N, dtype=dtype) if N % 2 else None
    layer = Linear(w, bias, act=act, out_dtype=out_dtype)
    ref = R.linear_backward(*d64(x, w, z, dout), act, dtype, out_dtype, gd)
    outs = layer.backward(x, dout, z=z, w_grad_dtype=gd)
    for name, got in zip(("dx", "dw", "dbias"), outs):
        if name == "dbias" and bias is None:
            assert got is None
        else:
            R.check(name, got, ref[name])
    again = layer.backward(x, dout, z=z, w_grad_dtype=gd)
    assert all(p is None or torch.equal(p, q) for p, q in zip(outs, again)), "two calls differ"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,I,pad,shift", [(3, 64, 40, 8, 0), (33, 128, 72, 8, 8), (70, 96, 136, 3, 1), (9, 65, 31, 1, 1),
                                             (130, 256, 128, 64, 64), (20, 40, 24, 7, 5)])
def test_strides_and_alignment(T, d, I, pad, shift, dt):
    """Rows further apart than they are long, starting anywhere: the gaps (NaN)
    are neither read nor written."""
    say(f"case: strides T {T} d {d} I {I} pad {pad} shift {shift} {dt}")
    dtype = DT[dt]
    vals = dict(x=rand(1, T, d, dtype=dtype), wg=rand(2, I, d, std=d ** -.5, dtype=dtype),
                wu=rand(3, I, d, std=d ** -.5, dtype=dtype), a=rand(6, T, I, dtype=dtype), b=rand(7, T, I, dtype=dtype),
                dh=rand(8, T, I, std=.1, dtype=dtype), wd=rand(9, d, I, std=I ** -.5, dtype=dtype),
                res=rand(10, T, d, dtype=dtype))
    v = {k: strided(t, pad, shift)[0] for k, t in vals.items()}
    layer = GatedProjection(v["wg"], v["wu"], act="silu")
    h, hbuf = strided(torch.zeros(T, I, dtype=dtype, device="cuda"), pad, shift)
    layer.forward(v["x"], out=h)
    R.check("h", h, R.gated_forward(*d64(vals["x"], vals["wg"], vals["wu"]), None, None, "silu", dtype)["h"])
    assert int(hbuf.isnan().sum()) == hbuf.numel() - T * I, "something beside h was written"
    dx, dxbuf = strided(torch.zeros(T, d, dtype=dtype, device="cuda"), pad, shift)
    outs = layer.backward(v["x"], v["a"], v["b"], v["dh"], dx=dx)
    ref = R.gated_backward(*d64(*(vals[k] for k in ("x", "wg", "wu", "a", "b", "dh"))), "silu", dtype, dtype)
    for name, got in zip(("dx", "dw_gate", "dw_up"), outs):
        R.check(name, got, ref[name])
    assert int(dxbuf.isnan().sum()) == dxbuf.numel() - T * d, "something beside dx was written"
    lin = Linear(v["wd"])
    y, ybuf = strided(torch.zeros(T, d, dtype=dtype, device="cuda"), pad, shift)
    lin.forward(v["dh"], residual=v["res"], out=y)
    R.check("y", y, R.linear_forward(*d64(vals["dh"], vals["wd"]), None, "none", vals["res"].double(), dtype, dtype)["y"])
    assert int(ybuf.isnan().sum()) == ybuf.numel() - T * d, "something beside y was written"
    outs = lin.backward(v["dh"], v["res"])
    ref = R.linear_backward(*d64(vals["dh"], vals["wd"]), None, vals["res"].double(), "none", dtype, dtype, dtype)
    for name, got in zip(("dx", "dw"), outs):
        R.check(name, got, ref[name])


@pytest.mark.parametrize("dt", DT)
def test_no_tokens(dt):
    dtype = DT[dt]
    wg, wu, bias = rand(2, 40, 64, dtype=dtype), rand(3, 40, 64, dtype=dtype), rand(4, 40, dtype=dtype)
    none = torch.empty(0, 64, dtype=dtype, device="cuda")
    empty = torch.empty(0, 40, dtype=dtype, device="cuda")
    g = GatedProjection(wg, wu, bias, bias)
    assert g.forward(none).shape == (0, 40)
    dx, *rest = g.backward(none, empty, empty, empty)
    assert dx.shape == (0, 64) and all(not t.any() and t.isfinite().all() for t in rest)
    lin = Linear(wg, bias, act="gelu")
    assert lin.forward(none).shape == (0, 40)
    dx, dw, db = lin.backward(none, empty, z=empty)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.isfinite().all() and db.isfinite().all()


@pytest.mark.parametrize("T", [1, 5, 16, 40, 200])
@pytest.mark.parametrize("dt", DT)
def test_special_values_stay_in_their_row(dt, T):
    """An infinity or NaN in one token's row, or one weight's row, spoils what it
    is part of and nothing else."""
    say(f"case: special values T {T} {dt}")
    dtype, d, I = DT[dt], 136, 72
    x, wg, wu = rand(1, T, d, dtype=dtype), rand(2, I, d, std=d ** -.5, dtype=dtype), rand(3, I, d, std=d ** -.5, dtype=dtype)
    clean = GatedProjection(wg, wu).forward(x)
    ylin = Linear(wg, out_dtype=torch.float32).forward(x)
    for bad in (float("nan"), float("inf"), float("-inf")):
        xb = x.clone()
        xb[T // 2, 5] = bad
        h, y = GatedProjection(wg, wu).forward(xb), Linear(wg, out_dtype=torch.float32).forward(xb)
        rows = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(h[rows], clean[rows]) and torch.equal(y[rows], ylin[rows])
        if bad != bad:
            assert h[T // 2].isnan().all() and y[T // 2].isnan().all()
        else:  # an infinity times a weight that is not zero
            want = torch.where(wg[:, 5] > 0, bad, -bad).float()
            want[wg[:, 5] == 0] = float("nan")
            assert torch.equal(y[T // 2][wg[:, 5] != 0], want[wg[:, 5] != 0])
        wb = wg.clone()
        wb[7, 3] = bad
        h = GatedProjection(wb, wu).forward(x)
        cols = torch.arange(I, device="cuda") != 7
        assert torch.equal(h[:, cols], clean[:, cols])
        if bad != bad:
            assert h[:, 7].isnan().all()
        # backward: dx keeps to the row, dW to the column of x
        a, b, dh = rand(6, T, I, dtype=dtype), rand(7, T, I, dtype=dtype), rand(8, T, I, std=.1, dtype=dtype)
        g = GatedProjection(wg, wu)
        c, s = g.backward(x, a, b, dh), g.backward(xb, a, b, dh)
        assert torch.equal(c[0], s[0])
        cols = torch.arange(d, device="cuda") != 5
        assert torch.equal(c[1][:, cols], s[1][:, cols]) and torch.equal(c[2][:, cols], s[2][:, cols])
        assert not s[1][:, 5].isfinite().any()
        dhb = dh.clone()
        dhb[T // 2, 9] = bad
        s = g.backward(x, a, b, dhb)
        assert torch.equal(c[0][rows], s[0][rows])
        keep = torch.arange(I, device="cuda") != 9
        assert torch.equal(c[1][keep], s[1][keep]) and torch.equal(c[2][keep], s[2][keep])


@pytest.mark.parametrize("act", ACTS)
def test_activation_range(act):
    """Every activation and its derivative from -inf to inf, NaN included, through
    a product with the identity."""
    v = torch.cat([torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1e-40]),
                   torch.linspace(-30, 30, 441), torch.logspace(-6, 38, 60), -torch.logspace(-6, 38, 60)]).cuda()
    v = v[:, None].contiguous()
    one = torch.ones(1, 1, device="cuda")
    fin = v[:, 0].isfinite()
    y, z = Linear(one, act=act).forward(v, save=True)
    assert torch.equal(z[fin], v[fin])
    ref, slope = R.act_both(v.double(), act)
    ok = (y.double() - ref).abs() <= ref.abs() * (R.act_rel(v.double().clamp(-40, 40)) + 2 ** -24) + 1e-37
    assert ok[fin].all(), v[fin][~ok[fin]]
    dx, _, = Linear(one, act=act).backward(v, torch.ones_like(v), z=v)[:2]
    tol = (1 + v.double().abs().clamp(max=40)) * (R.act_rel(v.double().clamp(-40, 40)) + 4 * R.EPS23)
    ok = (dx.double() - torch.where(v.double().abs() > 40, (v > 0).double() if act != "none" else 1.0, slope)).abs() <= tol
    assert ok[fin].all(), v[fin][~ok[fin]]
    inf, ninf, nan = (int(i) for i in (2, 3, 4))
    assert y[inf] == float("inf") and y[nan].isnan().all() and dx[nan].isnan().all() == (act != "none")
    assert y[ninf] == (float("-inf") if act == "none" else 0.0)
    assert dx[inf] == 1.0 and dx[ninf] == (1.0 if act == "none" else 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_past_32_bits(dt):
    """Outputs, saved sums and dz longer than 2^32 bytes (bf16: 2^31 elements too)."""
    dtype, K, N = DT[dt], 24, 8192
    T = 300_000 if dt == "bf16" else 140_000
    say(f"case: long offsets T {T} N {N} {dt}")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -.5).to(dtype)
    y, z = Linear(w, act="silu").forward(x, save=True)
    rows = torch.tensor([0, 1, T // 3, 131_071, 131_072, 131_073, T - 2, T - 1], device="cuda")
    ref = R.linear_forward(*d64(x[rows], w), None, "silu", None, dtype, dtype)
    R.check("y", y[rows], ref["y"])
    R.check("z", z[rows], ref["z"])
    dx, dw, _ = Linear(w, act="silu").backward(x, y, z=z, w_grad_dtype=torch.float32)
    cols = torch.tensor([0, 5, N - 1], device="cuda")
    zc, yc, xc = z[:, cols].double(), y[:, cols].double(), x.double()
    part = R.linear_backward(xc, w[cols].double(), zc, yc, "silu", dtype, dtype, torch.float32)
    R.check("dw", dw[cols], part["dw"])
    del zc, yc, xc, part
    ref = R.linear_backward(*d64(x[rows], w, z[rows], y[rows]), "silu", dtype, dtype, torch.float32)
    R.check("dx", dx[rows], ref["dx"])


@pytest.mark.parametrize("T,d,I,dt", [(1, 64, 48, "bf16"), (16, 256, 128, "bf16"), (100, 136, 72, "f16"), (70, 65, 33, "f32"),
                                      (300, 512, 256, "bf16")])
def test_graph_and_streams(T, d, I, dt):
    """Both operators, forward and backward, captured once and replayed with new
    inputs between eager work; two graphs replayed on two streams at once."""
    say(f"case: graph T {T} d {d} I {I} {dt}")
    dtype = DT[dt]
    wg, wu, wd = (rand(s, *sh, std=.1, dtype=dtype) for s, sh in ((2, (I, d)), (3, (I, d)), (4, (d, I))))
    bias = rand(5, I, dtype=dtype)
    gp, lin = GatedProjection(wg, wu, bias, bias), Linear(wd, out_dtype=torch.float32)

    def step(x, dy):
        h, a, b = gp.forward(x, save=True)
        y = lin.forward(h, residual=dy)
        dh, dwd, _ = lin.backward(h, dy)
        return (h, y, dh, dwd) + gp.backward(x, a, b, dh)

    xs = [rand(20 + i, T, d, dtype=dtype) for i in range(4)]
    dys = [rand(30 + i, T, d) for i in range(4)]
    want = [step(x, dy) for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        sx, sdy = xs[0].clone(), dys[0].clone()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            step(sx, sdy)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = step(sx, sdy)
        graphs.append((g, sx, sdy, outs))
    for i in (0, 1, 2, 3, 1):
        for g, sx, sdy, outs in graphs[:1]:
            sx.copy_(xs[i])
            sdy.copy_(dys[i])
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(outs, want[i])), f"replay of input {i} differs"
            again = step(xs[(i + 1) % 4], dys[(i + 1) % 4])  # eager work between replays
            assert all(torch.equal(p, q) for p, q in zip(again, want[(i + 1) % 4]))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for k, (g, sx, sdy, outs) in enumerate(graphs):
        sx.copy_(xs[k + 1])
        sdy.copy_(dys[k + 1])
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, *_), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for k, (g, sx, sdy, outs) in enumerate(graphs):
        assert all(torch.equal(p, q) for p, q in zip(outs, want[k + 1])), "graphs replayed side by side differ"
    # eager calls of one object on two streams at once
    got = []
    for k, s in enumerate((s1, s2)):
        with torch.cuda.stream(s):
            for _ in range(4):
                got.append((k, step(xs[k], dys[k])))
    torch.cuda.synchronize()
    for k, outs in got:
        assert all(torch.equal(p, q) for p, q in zip(outs, want[k])), "calls on two streams differ"


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_block_gradients_against_differences(act):
    """A feed-forward block y = x' + W_down gated(x) in fp32, forward and backward
    through both operators, against central differences of its 64-bit form."""
    T, d, I = 37, 48, 40
    x, dy = rand(1, T, d), rand(2, T, d)
    wg, wu, wd = rand(3, I, d, std=d ** -.5), rand(4, I, d, std=d ** -.5), rand(5, d, I, std=I ** -.5)
    bg, bu, bd = rand(6, I, std=.1), rand(7, I, std=.1), rand(8, d, std=.1)
    gp, lin = GatedProjection(wg, wu, bg, bu, act=act), Linear(wd, bd)
    h, a, b = gp.forward(x, save=True)
    dh, dwd, dbd = lin.backward(h, dy)
    dx, dwg, dwu, dbg, dbu = gp.backward(x, a, b, dh)
    grads = [dx + dy, dwg, dwu, dbg, dbu, dwd, dbd]
    params = d64(x, wg, wu, bg, bu, wd, bd)

    def loss(x, wg, wu, bg, bu, wd, bd):
        h = R.act_both(x @ wg.t() + bg, act)[0] * (x @ wu.t() + bu)
        return float(((x + h @ wd.t() + bd) * dy.double()).sum())

    # Central differences of step e along a unit-scale direction are within e^2/6 times the third derivative
    # (of order |loss terms| here) plus 2^-52 |loss| / e: about 1e-8 and 1e-9 relative at e = 1e-4.  The
    # fp32 gradients are within 1e-5 of theirs (sums of at most 48 products).
    e = 1e-4
    for i, g in enumerate(grads):
        v = rand(50 + i, *g.shape).double()
        lo, hi = list(params), list(params)
        lo[i], hi[i] = params[i] - e * v, params[i] + e * v
        num = (loss(*hi) - loss(*lo)) / (2 * e)
        ana = float((g.double() * v).sum())
        scale = float((g.double() * v).norm()) + 1e-9
        assert abs(num - ana) <= 1e-4 * scale, (i, num, ana, scale)


@pytest.mark.parametrize("T", [1, 16, 300])
def test_shared_expert_beside_the_moe_layer(T):
    """The use these operators are for: a shared expert beside routed ones.  The
    gated projection and the linear layer write x' + shared(x) in fp32, which the
    MoE layer takes as its residual."""
    say(f"case: shared expert beside the layer, T {T}")
    cfg = syn.gen.Config(190, "shared", (T,), 512, 8, 256, 2, "bf16", "bf16", "router")
    case = Case(cfg, T)
    x = case.x.cuda()
    wg, wu = rand(41, 384, 512, std=512 ** -.5, dtype=torch.bfloat16), rand(42, 384, 512, std=512 ** -.5, dtype=torch.bfloat16)
    wd = rand(43, 512, 384, std=384 ** -.5, dtype=torch.bfloat16)
    stream = rand(44, T, 512)
    h = GatedProjection(wg, wu).forward(x)
    run = stream.clone()
    Linear(wd, out_dtype=torch.float32).forward(h, residual=run, out=run)
    href = R.gated_forward(*d64(x, wg, wu), None, None, "silu", torch.bfloat16)["h"]
    y, bound = R.product(href[0], wd.double(), href[1])
    shared = (stream.double() + y, bound + (stream.double() + y).abs() * 2.0 ** -23)
    R.check("shared", run, shared)
    alone = case.run()["out"]
    both = case.run(residual=run)["out"]
    # the layer adds its residual to the finished sum: one fp32 rounding
    want = alone.astype(np.float64) + run.double().cpu().numpy()
    assert np.all(np.abs(both - want) <= np.abs(want) * 2.0 ** -23 + 1e-30)


def test_another_device_is_refused_or_served():
    """Tensors must share the weights' device; a call made while another device
    is current runs on the weights' own."""
    w = rand(1, 8, 16)
    with pytest.raises(ValueError):
        Linear(w).forward(torch.zeros(2, 16))
    if torch.cuda.device_count() > 1:
        x = rand(2, 3, 16)
        want = Linear(w).forward(x)
        with torch.cuda.device(1):
            assert torch.equal(Linear(w).forward(x), want)


def big(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# sizes at which a call takes the larger tiles, splits its reduction, streams the weights or joins its
# two backward products, with widths on and off the 16-byte chunks and the tiles
LARGE = [(4096, 1024, 2048), (2048, 4096, 4096), (1500, 2000, 1800), (1501, 1999, 1803), (700, 4096, 1030),
         (40, 4096, 1024), (64, 512, 768), (24, 1023, 1531), (12, 5001, 640), (9, 2048, 8200), (150, 7000, 260),
         (5000, 130, 96), (3001, 70, 1210), (18, 8192, 4112), (333, 1200, 5000)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", LARGE)
def test_larger_linear(T, K, N, dt):
    say(f"case: larger linear T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    x, w = big(1, T, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype)
    bias, residual = big(4, N, dtype=dtype), big(5, T, N, dtype=dtype)
    layer = Linear(w, bias, act="silu")
    ref = R.linear_forward(*d64(x, w, bias), "silu", residual.double(), dtype, dtype)
    y, z = layer.forward(x, residual=residual, save=True)
    R.check("z", z, ref["z"])
    R.check("y", y, ref["y"])
    assert torch.equal(layer.forward(x, residual=residual), y)
    del ref
    dout = big(8, T, N, std=0.1, dtype=dtype)
    ref = R.linear_backward(*d64(x, w, z, dout), "silu", dtype, dtype, dtype)
    outs = layer.backward(x, dout, z=z)
    for name, got in zip(("dx", "dw", "dbias"), outs):
        R.check(name, got, ref[name])
    assert all(torch.equal(p, q) for p, q in zip(outs, layer.backward(x, dout, z=z))), "two calls differ"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,I", LARGE)
def test_larger_gated(T, d, I, dt):
    say(f"case: larger gated T {T} d {d} I {I} {dt}")
    dtype = DT[dt]
    x, wg, wu = big(1, T, d, dtype=dtype), big(2, I, d, std=d ** -.5, dtype=dtype), big(3, I, d, std=d ** -.5, dtype=dtype)
    bg, bu = big(4, I, dtype=dtype), big(5, I, dtype=dtype)
    layer = GatedProjection(wg, wu, bg, bu, act="gelu")
    ref = R.gated_forward(*d64(x, wg, wu, bg, bu), "gelu", dtype)
    h, a, b = layer.forward(x, save=True)
    for name, got in (("h", h), ("a", a), ("b", b)):
        R.check(name, got, ref[name])
    assert torch.equal(layer.forward(x), h)
    del ref
    dh = big(8, T, I, std=0.1, dtype=dtype)
    ref = R.gated_backward(*d64(x, wg, wu, a, b, dh), "gelu", dtype, dtype)
    outs = layer.backward(x, a, b, dh)
    for name, got in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), outs):
        R.check(name, got, ref[name])
    assert all(torch.equal(p, q) for p, q in zip(outs, layer.backward(x, a, b, dh))), "two calls differ"


@pytest.mark.parametrize("T", [1, 3, 40, 300, 2000])
def test_fp32_magnitudes(T):
    """fp32 products over the whole range of exponents: near the largest values,
    far below bf16's rounding of them, and mixed within one sum."""
    say(f"case: fp32 magnitudes T {T}")
    K, N = 200, 150
    for scale_x, scale_w in ((1e30, 1e-30), (3e37, 1e-3), (1e-25, 1e20), (1e-36, 1.0)):
        x, w = rand(1, T, K) * scale_x, rand(2, N, K) * scale_w
        y = Linear(w).forward(x)
        ref, err = R.product(x.double(), w.double())
        R.check("y", y, (ref, err + R.half_step(ref, torch.float32) + K * 2.0 ** -134 * float(w.abs().max())))
    # rows of x of very different sizes stay apart
    x = rand(1, T, K) * torch.logspace(-30, 30, T, device="cuda")[:, None]
    w = rand(2, N, K)
    ref, err = R.product(x.double(), w.double())
    R.check("y", Linear(w).forward(x), (ref, err + R.half_step(ref, torch.float32)))


def test_out_of_place_partial_gradients():
    """The C entry points compute only what is asked for, and the same bits."""
    T, d, I = 100, 136, 72
    dt = torch.bfloat16
    x, wg, wu = rand(1, T, d, dtype=dt), rand(2, I, d, std=.1, dtype=dt), rand(3, I, d, std=.1, dtype=dt)
    a, b, dh, bias = rand(6, T, I, dtype=dt), rand(7, T, I, dtype=dt), rand(8, T, I, std=.1, dtype=dt), rand(4, I, dtype=dt)
    full = GatedProjection(wg, wu, bias, bias).backward(x, a, b, dh)
    ws = torch.empty(ecf.ecf_gated_workspace_bytes(d, I, ecf.ECF_BF16, T, True), dtype=torch.uint8, device="cuda")
    for want in (("dx",), ("dw",), ("db_up",), ("dx", "db_gate")):
        q = ecf.GatedArgs()
        q.hidden, q.inter, q.dtype, q.wgrad_dtype, q.act = d, I, ecf.ECF_BF16, ecf.ECF_BF16, ecf.ECF_ACT_SILU
        q.d_x, q.d_w_gate, q.d_w_up, q.d_a, q.d_b, q.d_dh = (t.data_ptr() for t in (x, wg, wu, a, b, dh))
        q.d_ws, q.ws_bytes = ws.data_ptr(), ws.numel()
        got = {k: torch.full_like(t, float("nan")) for k, t in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), full)}
        for k in want:
            for f in (("dw_gate", "dw_up") if k == "dw" else (k,)):
                setattr(q, "d_" + f, got[f].data_ptr())
        ecf.ecf_gated_backward(q, T)
        torch.cuda.synchronize()
        for k, t in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), full):
            asked = k in want or ("dw" in want and k.startswith("dw"))
            if asked:
                # another choice of tiles may add in another order: both are within the bound of one rounding
                R.check(k, got[k], (t.double(), 2 * R.half_step(t.double(), dt) + 1e-4))
            if not asked:
                assert got[k].isnan().all(), k


# one product at a time, at sizes that between them take every tile on both paths to LDS
ONE = [(4100, 2050, 4101), (4101, 1025, 4099), (1025, 1030, 2051), (600, 700, 1101), (300, 260, 521), (130, 100, 67),
       (4096, 4096, 4096), (4096, 1024, 4096), (2048, 2048, 2048), (1024, 1024, 2048), (512, 768, 640), (136, 128, 64)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", ONE)
def test_one_gradient_at_a_time(T, K, N, dt):
    say(f"case: one gradient T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    x, w, dout = big(1, T, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype), big(8, T, N, std=.1, dtype=dtype)
    bias = big(3, N, dtype=dtype)
    layer = Linear(w, bias)
    ref = R.linear_backward(*d64(x, w), None, dout.double(), "none", dtype, dtype, dtype)
    dx, dw, db = layer.backward(x, dout, need_dw=False)
    assert dw is None and db is None
    R.check("dx", dx, ref["dx"])
    dx, dw, db = layer.backward(x, dout, need_dx=False)
    assert dx is None
    R.check("dw", dw, ref["dw"])
    R.check("dbias", db, ref["dbias"])
    R.check("y", layer.forward(x), R.linear_forward(*d64(x, w, bias), "none", None, dtype, dtype)["y"])
    if N * K * T < 1 << 34:
        wu = big(4, N, K, std=K ** -.5, dtype=dtype)
        g = GatedProjection(w, wu)
        R.check("h", g.forward(x), R.gated_forward(*d64(x, w, wu), None, None, "silu", dtype)["h"])
        a, b = big(5, T, N, dtype=dtype), big(6, T, N, dtype=dtype)
        ref = R.gated_backward(*d64(x, w, wu, a, b, dout), "silu", dtype, dtype)
        R.check("dx", g.backward(x, a, b, dout, need_dw=False)[0], ref["dx"])
        outs = g.backward(x, a, b, dout, need_dx=False)
        assert outs[0] is None
        R.check("dw_gate", outs[1], ref["dw_gate"])
        R.check("dw_up", outs[2], ref["dw_up"])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", [(1, 1024, 4096), (6, 640, 1500), (12, 640, 1500), (14, 333, 2047), (20, 512, 3000), (30, 511, 2301),
                                   (50, 384, 1000), (64, 200, 300), (7, 2049, 1201), (16, 4096, 96), (3, 16, 5000),
                                   (16, 8200, 130), (9, 16384, 70), (2, 66000, 40), (40, 5, 300),
                                   (20, 7, 9000), (36, 40, 200000), (24, 40, 200000)])
def test_few_tokens(T, K, N, dt):
    """Every shape of the streaming kernel: rows per block, groups of tokens, odd rows."""
    say(f"case: few tokens T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    x, w, wu = big(1, T, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype), big(4, N, K, std=K ** -.5, dtype=dtype)
    bias, res = big(3, N, dtype=dtype), big(5, T, N)
    layer = Linear(w, bias, act="gelu_tanh", out_dtype=torch.float32)
    y, z = layer.forward(x, residual=res, save=True)
    ref = R.linear_forward(*d64(x, w, bias), "gelu_tanh", res.double(), dtype, torch.float32)
    R.check("y", y, ref["y"])
    R.check("z", z, ref["z"])
    h, a, b = GatedProjection(w, wu, None, bias, act="silu").forward(x, save=True)
    ref = R.gated_forward(*d64(x, w, wu), None, bias.double(), "silu", dtype)
    for name, got in (("h", h), ("a", a), ("b", b)):
        R.check(name, got, ref[name])


# M x N outputs over K, such that the estimates choose each tile in turn, with every width a multiple of 8
# (operands straight to LDS) and odd (through registers)
TILES = [(5264, 1584, 72), (136, 6416, 4088), (704, 6008, 72), (1296, 1744, 72), (72, 64, 80), (4736, 896, 72), (608, 3328, 72),
         (160, 5720, 72), (1055, 7703, 71), (3275, 263, 2407), (6957, 519, 75), (3195, 647, 71), (99, 71, 65), (1659, 2703, 67),
         (1111, 1819, 67), (5705, 171, 71), (6321, 71, 2661), (2047, 4093, 515)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", TILES)
def test_every_tile(M, N, K, dt):
    """One product shape in each place it can have: x W^T, gated, dz W and dz^T x."""
    say(f"case: tiles M {M} N {N} K {K} {dt}")
    dtype = DT[dt]
    a, b, b2 = big(1, M, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype), big(3, N, K, std=K ** -.5, dtype=dtype)
    ref = R.rounded(*R.product(a.double(), b.double()), dtype)
    R.check("x W^T", Linear(b).forward(a), ref)
    bt = b.t().contiguous()
    R.check("dz W", Linear(bt).backward(big(4, M, N, dtype=dtype), a, need_dw=False)[0], ref)
    at = a.t().contiguous()
    R.check("dz^T x", Linear(big(5, M, N, dtype=dtype)).backward(bt, at, need_dx=False)[1], ref)
    R.check("gated", GatedProjection(b, b2, act="none").forward(a),
            R.gated_forward(*d64(a, b, b2), None, None, "none", dtype)["h"])


def test_weights_given_other_memory():
    """w.data = ... leaves the object with the memory it was made on, which nothing else may get."""
    say("case: replaced weight memory")
    x, w = big(1, 40, 96), big(2, 64, 96, std=96 ** -.5)
    ref = R.linear_forward(*d64(x, w), None, "none", None, torch.float32, torch.float32)["y"]
    p = torch.nn.Parameter(w)
    layer = Linear(p)
    del w
    p.data = torch.zeros(64, 96, device="cuda")
    junk = [torch.full((64, 96), float("nan"), device="cuda") for _ in range(64)]
    R.check("y", layer.forward(x), ref)
    assert len(junk) == 64


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,I", [(65, 1, 5), (70, 5, 130), (200, 7, 64), (131, 20, 67), (300, 31, 200)])
def test_gated_short_rows(T, d, I, dt):
    """More tokens than are streamed, over rows under 8 elements (fp32: under 32)."""
    say(f"case: short rows T {T} d {d} I {I} {dt}")
    dtype = DT[dt]
    x, wg, wu = big(1, T, d, dtype=dtype), big(2, I, d, dtype=dtype), big(3, I, d, dtype=dtype)
    bg, bu = big(4, I, dtype=dtype), big(5, I, dtype=dtype)
    h, a, b = GatedProjection(wg, wu, bg, bu, act="gelu").forward(x, save=True)
    ref = R.gated_forward(*d64(x, wg, wu, bg, bu), "gelu", dtype)
    for name, got in (("h", h), ("a", a), ("b", b)):
        R.check(name, got, ref[name])
    da, db = big(6, T, I, dtype=dtype), big(7, T, I, dtype=dtype)
    dh = big(8, T, I, std=.1, dtype=dtype)
    outs = GatedProjection(wg, wu, bg, bu, act="gelu").backward(x, da, db, dh)
    ref = R.gated_backward(*d64(x, wg, wu, da, db, dh), "gelu", dtype, dtype)
    for name, got in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), outs):
        R.check(name, got, ref[name])


def wide(seed, rows, cols, dtype, std=1.0):
    """Rows of normal values, made a part at a time."""
    t = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for i, part in enumerate(t.split(8192)):
        part.copy_(big(seed * 1000 + i, *part.shape, std=std))
    return t


@pytest.mark.parametrize("K,N", [(16, 32768), (17, 32769), (5, 32768)])
def test_offsets_past_32_bits_in_outputs_and_gradients(K, N):
    """70000 x 32768 elements pass 2^31: rows at both ends and at the border, for every kind of kernel."""
    T, dtype = 70000, torch.bfloat16
    border = (1 << 31) // N
    rows = torch.tensor([0, 1, border - 1, border, border + 1, border + 2, T - 2, T - 1], device="cuda")
    cols = torch.tensor([0, 7, 63, 64, N // 2, N - 9, N - 2, N - 1], device="cuda")
    say(f"case: past 32 bits K {K} N {N}: forward")
    x, w, bias = big(1, T, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype), big(3, N, dtype=dtype)
    acc = wide(4, T, N, dtype)
    before = acc[rows].double()
    layer = Linear(w, bias, act="relu")
    y, z = layer.forward(x, residual=acc, out=acc, save=True)
    assert y is acc
    ref = R.linear_forward(x[rows].double(), *d64(w, bias), "relu", before, dtype, dtype)
    R.check("y", y[rows], ref["y"])
    R.check("z", z[rows], ref["z"])
    say("   backward")
    dx, dw, db = layer.backward(x, y, z, w_grad_dtype=torch.float32)
    ref = R.linear_backward(x[rows].double(), w.double(), z[rows].double(), y[rows].double(), "relu", dtype, dtype, torch.float32)
    R.check("dx", dx[rows], ref["dx"])
    ref = R.linear_backward(x.double(), w[cols].double(), z[:, cols].double(), y[:, cols].double(), "relu", dtype, dtype,
                            torch.float32)
    R.check("dw", dw[cols], ref["dw"])
    R.check("dbias", db[cols], ref["dbias"])
    del acc, y, z
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [3, 40])
def test_offsets_past_32_bits_in_weights(T):
    """Weights of 40000 x 60000 elements: streamed and in tiles, and as an operand of dx."""
    say(f"case: past 32 bits in weights T {T}")
    N, K, dtype = 40000, 60000, torch.bfloat16
    w = wide(5, N, K, dtype, std=K ** -.5)
    x = big(6, T, K, dtype=dtype)
    cols = torch.tensor([0, 1, 15, 16, (1 << 31) // K - 1, (1 << 31) // K, (1 << 31) // K + 1, N - 2, N - 1], device="cuda")
    layer = Linear(w)
    y = layer.forward(x)
    R.check("y", y[:, cols], R.linear_forward(x.double(), w[cols].double(), None, "none", None, dtype, dtype)["y"])
    # rows of dout that touch these weight rows only: dx is a sum of theirs
    dout = torch.zeros(T, N, dtype=dtype, device="cuda")
    dout[:, cols] = big(7, T, len(cols), dtype=dtype)
    dx = layer.backward(x, dout, need_dw=False)[0]
    ref = R.linear_backward(x.double(), w[cols].double(), None, dout[:, cols].double(), "none", dtype, dtype, dtype)
    R.check("dx", dx, ref["dx"])
    dw = layer.backward(x, dout, need_dx=False)[1]
    R.check("dw", dw[cols], ref["dw"])
    del w, dw
    torch.cuda.empty_cache()
