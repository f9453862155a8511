"""GPU tests of the norm with the residual's addition against the 64-bit reference of
tokens_ref.py: types, row lengths around every kernel's border, strides and alignment, the 8-bit
output, special values, in-place sums, the gradients."""
import pytest
import torch

import dense_ref as R
import expert_cache_ffn_amd as ecf
import tokens_ref as TR
from expert_cache_ffn_amd.layer import RMSNorm
from gpu_util import say
from tokens_ref import DT, rand, strided

pytestmark = pytest.mark.gpu

# (tokens, d): rows of one element, off the vector width, around each length where another kernel takes over
SIZES = [(1, 1), (3, 7), (2, 8), (5, 31), (4, 33), (1, 512), (9, 513), (6, 1000), (3, 1024), (5, 1025), (2, 2048), (7, 2731),
         (1, 4096), (33, 4096), (4, 4100), (3, 8192), (2, 8200), (3, 16384), (2, 16385), (1, 16392), (2, 40007), (517, 64),
         (1100, 129), (2, 16400), (9000, 24)]
EPS = 1e-6


def inputs(T, d, dt, sum_dt, seed=0):
    dtype, st = DT[dt], DT[sum_dt]
    return rand(seed + 1, T, d, dtype=dtype), rand(seed + 2, T, d, std=2.0, dtype=st), (1 + rand(seed + 3, d, std=0.2).double()).to(dtype)


@pytest.mark.parametrize("dt,sum_dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("T,d", SIZES)
def test_forward(T, d, dt, sum_dt):
    say(f"case: norm forward T {T} d {d} {dt} sum {sum_dt}")
    x, res, w = inputs(T, d, dt, sum_dt)
    norm = RMSNorm(w, eps=EPS, sum_dtype=DT[sum_dt])
    for residual in (res, None):
        total = TR.norm_sum(x, residual)
        ref = TR.norm_forward(total, w, EPS, DT[dt])
        o = norm.forward(x, residual=residual, mx=True, save=True)
        assert torch.equal(o.sum, total) and (residual is not None or o.sum is x)
        R.check("y", o.y, ref["y"])
        R.check("rstd", o.rstd, ref["rstd"])
        assert o.q.shape == (T, d) and o.scale.shape == (T, (d + 31) // 32)
        TR.check_mx(o.q, o.scale, ref["exact"])
        again = norm.forward(x, residual=residual)
        assert torch.equal(again.y, o.y) and again.rstd is None and again.q is None
        only = norm.forward(x, residual=residual, y=False, mx=True)
        assert only.y is None and torch.equal(only.q.view(torch.uint8), o.q.view(torch.uint8))
    kept = res.clone()
    o = norm.forward(x, residual=kept, sum_out=kept)
    assert o.sum is kept and torch.equal(kept, TR.norm_sum(x, res)) and torch.equal(o.y, norm.forward(x, residual=res).y)


@pytest.mark.parametrize("dt,sum_dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("T,d", SIZES)
def test_backward(T, d, dt, sum_dt):
    say(f"case: norm backward T {T} d {d} {dt} sum {sum_dt}")
    dtype, st = DT[dt], DT[sum_dt]
    _, total, w = inputs(T, d, dt, sum_dt)
    dy, dsum = rand(5, T, d, std=0.1, dtype=dtype), rand(6, T, d, std=0.1, dtype=st) if d % 3 else None
    norm = RMSNorm(w, eps=EPS, sum_dtype=st)
    rstd = TR.norm_forward(total, w, EPS, dtype)["rstd"][0].float()
    gd = torch.float32 if T % 2 else dtype
    ref = TR.norm_backward(total, rstd, w, dy, dsum, dtype, st, gd)
    dx, ds, dw = norm.backward(total, rstd, dy, dsum=dsum, w_grad_dtype=gd)
    assert (dx is ds) == (dtype is st)
    for name, got in (("dx", dx), ("ds", ds), ("dw", dw)):
        R.check(name, got, ref[name])
    if dsum is not None:  # in place
        kept = dsum.clone()
        dx2, ds2, none = norm.backward(total, rstd, dy, dsum=kept, ds=kept, need_dw=False)
        assert ds2 is kept and none is None and torch.equal(ds2, ds) and torch.equal(dx2, dx)
    none, none2, dw2 = norm.backward(total, rstd, dy, dsum=dsum, w_grad_dtype=gd, need_dx=False)
    assert none is None and none2 is None and torch.equal(dw2, dw)


def test_weight_types_and_none():
    x, res, w = inputs(5, 200, "bf16", "f32")
    norm = RMSNorm(w.float(), dtype=torch.bfloat16, sum_dtype=torch.float32)
    ref = TR.norm_forward(TR.norm_sum(x, res), w, 1e-6, torch.bfloat16)
    o = norm.forward(x, residual=res, save=True)
    R.check("y", o.y, ref["y"])
    dy = rand(5, 5, 200, dtype=torch.bfloat16)
    dx, ds, dw = norm.backward(o.sum, o.rstd, dy)
    back = TR.norm_backward(o.sum, o.rstd, w, dy, None, torch.bfloat16, torch.float32, torch.float32)
    for name, got in (("dx", dx), ("ds", ds), ("dw", dw)):
        R.check(name, got, back[name])
    assert dw.dtype is torch.float32
    # an x without a residual beside an fp32 stream: its gradient has its own type
    o = norm.forward(x, save=True)
    dx, ds, _ = norm.backward(o.sum, o.rstd, dy)
    assert dx is ds and dx.dtype is torch.bfloat16
    # no weight: ones (C ABI)
    a = ecf.NormArgs()
    a.hidden, a.eps = 200, 1e-6
    y = torch.empty_like(x)
    a.dtype = a.sum_dtype = a.weight_dtype = ecf.ECF_BF16
    a.d_x, a.d_y = x.data_ptr(), y.data_ptr()
    ecf.ecf_norm_forward(a, 5)
    torch.cuda.synchronize()
    R.check("y", y, TR.norm_forward(x, None, 1e-6, torch.bfloat16)["y"])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d,pad,shift", [(3, 100, 5, 1), (4, 264, 1, 3), (2, 9000, 7, 2), (5, 4096, 3, 1), (2, 20000, 9, 5)])
def test_strides(T, d, pad, shift, dt):
    say(f"case: norm strides T {T} d {d} pad {pad} shift {shift} {dt}")
    dtype = DT[dt]
    x, res, w = inputs(T, d, dt, dt)
    norm = RMSNorm(w)
    xs, rs = strided(x, pad, shift)[0], strided(res, pad + 1, shift + 1)[0]
    out, out_buf = strided(torch.zeros_like(x), pad + 2, shift)
    total, total_buf = strided(torch.zeros_like(x), pad + 3, shift)
    want = norm.forward(x, residual=res, save=True)
    o = norm.forward(xs, residual=rs, out=out, sum_out=total)
    assert torch.equal(o.y, want.y) and torch.equal(o.sum, want.sum)
    for buf, ld in ((out_buf, d + pad + 2), (total_buf, d + pad + 3)):  # the gaps are as they were
        assert torch.isnan(buf[:shift]).all() and torch.isnan(buf[shift:].view(T, ld)[:, d:]).all()
    dy, dsum = rand(5, T, d, dtype=dtype), rand(6, T, d, dtype=dtype)
    want_b = norm.backward(want.sum, want.rstd, dy, dsum=dsum)
    ds, ds_buf = strided(torch.zeros_like(x), pad, shift)
    got_b = norm.backward(o.sum, want.rstd, strided(dy, pad, shift + 1)[0], dsum=strided(dsum, 1, 1)[0], ds=ds)
    for p, q in zip(got_b, want_b):
        assert torch.equal(p, q)
    assert torch.isnan(ds_buf[shift:].view(T, d + pad)[:, d:]).all()


def test_8_bit_values():
    """The 8-bit output is the fp32 one in e4m3 to the bit, scales by the definition: every magnitude, ties, zeros, NaN."""
    g = torch.Generator().manual_seed(3)
    T, d = 64, 320
    # eps so large that rstd is one power of two: y takes the values of x
    x = torch.randn(T, d, generator=g, dtype=torch.float64).float()
    x[0] = 0
    x[1, :32] = 2.0 ** -140
    x[2] = torch.ldexp(torch.randint(-127, 128, (d,), generator=g).float(), torch.tensor(-6))
    x[3, 7] = 448.0
    x[4, :32] = torch.tensor([448.0] + [16.0 * i + 1.0 * (i % 3) for i in range(1, 28)] + [8.5, 9.0, 9.5, 2.0 ** -9])
    x[5] *= 1e-30
    x = x.cuda()
    norm = RMSNorm(torch.ones(d, device="cuda"), eps=4.0 ** 40)
    o = norm.forward(x, mx=True)
    b = TR.mx_bytes(o.y)
    assert torch.equal(o.scale.view(torch.uint8).long(), b.long())
    want = (o.y.double() * torch.exp2(127 - b.double()).repeat_interleave(32, dim=1)).float().to(torch.float8_e4m3fn)
    assert torch.equal(o.q.view(torch.uint8), want.view(torch.uint8))


def test_special_values():
    """A row's infinities and NaN stay in it; rows of zeros, of the largest and of tiny values."""
    for dt in DT:
        T, d = 6, 300
        x, res, w = inputs(T, d, dt, dt)
        clean = RMSNorm(w).forward(x, mx=True)
        bad = x.clone()
        bad[1, 5], bad[3, 299] = float("nan"), float("inf")
        bad[4] = 0
        o = RMSNorm(w).forward(bad, mx=True, save=True)
        for t in (0, 2, 5):
            assert torch.equal(o.y[t], clean.y[t]) and torch.equal(o.q.view(torch.uint8)[t], clean.q.view(torch.uint8)[t])
        assert torch.isnan(o.y[1]).all() and torch.isnan(o.q[1].float()).all()
        assert torch.isnan(o.y[3, 299]) and (o.y[3, :299] == 0).all() and torch.isnan(o.q[3, 299].float())
        assert (o.y[4] == 0).all() and (o.q[4].float() == 0).all() and (o.scale[4].view(torch.uint8) == 0).all()
    for big in (1e30, 1e-30):  # squares outside fp32's range
        x = rand(1, 4, 300, std=big)
        ref = TR.norm_forward(x, None, 0.0, torch.float32)
        o = RMSNorm(torch.ones(300, device="cuda"), eps=0.0).forward(x, save=True)
        R.check("y", o.y, ref["y"])
        R.check("rstd", o.rstd, ref["rstd"])


def test_no_tokens():
    w = torch.ones(40, device="cuda")
    norm = RMSNorm(w)
    x = torch.empty(0, 40, device="cuda")
    o = norm.forward(x, residual=x, mx=True, save=True)
    assert o.y.shape == o.sum.shape == o.q.shape == (0, 40) and o.scale.shape == (0, 2)
    dx, ds, dw = norm.backward(o.sum, o.rstd, x)
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros_like(dw))


def test_gradient_against_differences():
    x, res, w = rand(1, 4, 50), rand(2, 4, 50), 1 + rand(3, 50, std=0.1)
    norm = RMSNorm(w, eps=1e-3)
    dy, dsum = rand(4, 4, 50), rand(5, 4, 50)

    def loss(r):
        s = x.double() + r
        return ((s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-3) * w.double()) * dy.double()).sum() + (s * dsum.double()).sum()

    o = norm.forward(x, residual=res, save=True)
    _, ds, _ = norm.backward(o.sum, o.rstd, dy, dsum=dsum)
    step = rand(6, 4, 50).double()
    h = 1e-4
    slope = (loss(res.double() + h * step) - loss(res.double() - h * step)) / (2 * h)
    assert abs(float((ds.double() * step).sum() - slope)) <= 1e-4 * abs(float(slope)) + 1e-4


def test_graph_and_streams():
    x, res, w = inputs(64, 1000, "bf16", "f32")
    norm = RMSNorm(w, sum_dtype=torch.float32)
    dy = rand(5, 64, 1000, dtype=torch.bfloat16)

    def step():
        o = norm.forward(x, residual=res, mx=True, save=True)
        return [o.y, o.sum, o.q.view(torch.uint8), o.scale.view(torch.uint8), *norm.backward(o.sum, o.rstd, dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = step()
    torch.cuda.synchronize()
    for seed in range(4):
        x.copy_(rand(10 + seed, 64, 1000, dtype=torch.bfloat16))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(kept, want):
            assert torch.equal(p, q)
