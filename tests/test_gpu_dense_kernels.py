"""GPU tests of dense calls that reach kernels or operands the other files do not."""
import warnings

import pytest
import torch

import dense_ref as R
from expert_cache_ffn_amd.layer import GatedProjection, Linear
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# dW alone, over enough tokens to split them
SPLIT_DW = [(5000, 130, 96), (8001, 71, 65)]


def big(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", SPLIT_DW)
def test_split_weight_gradients_alone(T, K, N, dt):
    say(f"case: split weight gradients T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    x, dout = big(1, T, K, dtype=dtype), big(2, T, N, std=.1, dtype=dtype)
    w, z = big(3, N, K, dtype=dtype), big(4, T, N, dtype=dtype)
    ref = R.linear_backward(x.double(), w.double(), z.double(), dout.double(), "silu", dtype, dtype, torch.float32)
    layer = Linear(w, big(5, N, dtype=dtype), act="silu")
    dx, dw, db = layer.backward(x, dout, z, w_grad_dtype=torch.float32, need_dx=False)
    assert dx is None
    R.check("dw", dw, ref["dw"])
    R.check("dbias", db, ref["dbias"])
    assert torch.equal(layer.backward(x, dout, z, w_grad_dtype=torch.float32, need_dx=False)[1], dw)


@pytest.mark.parametrize("dt", DT)
def test_gradients_of_the_widest_layers(dt):
    """inter at the longest rows that are served: da and db lie in rows as long as dh's."""
    dtype = DT[dt]
    T, d, I = 5, 8, ((1 << 31) - 1) // 256 // dtype.itemsize
    say(f"case: widest gated backward T {T} d {d} I {I} {dt}")
    x, wg, wu = big(1, T, d, dtype=dtype), big(2, I, d, std=.1, dtype=dtype), big(3, I, d, std=.1, dtype=dtype)
    a, b, dh = big(4, T, I, dtype=dtype), big(5, T, I, dtype=dtype), big(6, T, I, std=.01, dtype=dtype)
    outs = GatedProjection(wg, wu, wg[:, 0].contiguous(), wu[:, 0].contiguous()).backward(x, a, b, dh)
    ref = R.gated_backward(*(t.double() for t in (x, wg, wu, a, b, dh)), "silu", dtype, dtype)
    for name, got in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), outs):
        R.check(name, got, ref[name])
    dx, dw, db = Linear(wg, act="gelu").backward(x, dh, a)
    ref = R.linear_backward(*(t.double() for t in (x, wg, a, dh)), "gelu", dtype, dtype, dtype)
    R.check("dx", dx, ref["dx"])
    R.check("dw", dw, ref["dw"])


# few tokens of wide layers, whose 16-bit rows at odd elements go through tiles without a workspace
ODD_ROWS = [("linear_forward", 13, 2046, 34967), ("linear_forward", 1, 4080, 56412), ("linear_forward", 16, 438, 23179),
            ("gated_forward", 16, 4096, 8192), ("gated_forward", 8, 1392, 24321), ("gated_forward", 13, 2334, 6332)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1)])
@pytest.mark.parametrize("op,T,K,N", ODD_ROWS)
def test_few_tokens_of_rows_at_odd_elements(op, T, K, N, pad, shift, dt):
    say(f"case: odd rows {op} T {T} K {K} N {N} pad {pad} shift {shift} {dt}")
    dtype = DT[dt]

    def rows(seed, r, std):
        v = big(seed, r * (K + pad) + shift, std=std, dtype=dtype)
        return v[shift:].view(r, K + pad)[:, :K]

    x, w, bias = rows(1, T, 1.0), rows(2, N, K ** -.5), big(3, N, dtype=dtype)
    if op == "linear_forward":
        y, z = Linear(w, bias, act="gelu").forward(x, save=True)
        ref = R.linear_forward(x.double(), w.double(), bias.double(), "gelu", None, dtype, dtype)
        R.check("y", y, ref["y"])
        R.check("z", z, ref["z"])
        return
    wu = rows(4, N, K ** -.5)
    h, a, b = GatedProjection(w, wu, bias).forward(x, save=True)
    ref = R.gated_forward(x.double(), w.double(), wu.double(), bias.double(), None, "silu", dtype)
    for name, got in (("h", h), ("a", a), ("b", b)):
        R.check(name, got, ref[name])


def test_a_forward_pass_that_loses_gradients_says_so():
    """Outputs carry no gradient function; a call whose caller would miss one warns, and gives the same bits."""
    x, w = big(1, 70, 96), big(2, 64, 96, std=.1)
    plain = Linear(w).forward(x), GatedProjection(w, w).forward(x)
    p = torch.nn.Parameter(w)
    lin, gp = Linear(p), GatedProjection(p, p)
    for f, want in ((lin.forward, plain[0]), (gp.forward, plain[1])):
        with pytest.warns(UserWarning, match="outside autograd"):
            y = f(x)
        assert torch.equal(y, want) and y.grad_fn is None
        with pytest.warns(UserWarning, match="outside autograd"):
            f(x.clone().requires_grad_())
    with pytest.warns(UserWarning, match="outside autograd"):
        Linear(w).forward(x, residual=torch.zeros(70, 64, device="cuda", requires_grad=True))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            assert torch.equal(lin.forward(x), plain[0])
        assert torch.equal(lin.forward(x, save=True)[0], plain[0])  # for backward()
        assert torch.equal(gp.forward(x, save=True)[0], plain[1])
        assert torch.equal(Linear(w).forward(x), plain[0])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,K,N", [(8192, 640, 1), (5000, 333, 3), (4099, 72, 7), (6000, 1, 200), (5001, 7, 129), (9000, 5, 6)])
def test_narrow_layers_over_many_tokens(T, K, N, dt):
    """Rows of under 8 elements with reductions of thousands: a head of a few outputs, a layer of a few inputs."""
    say(f"case: narrow T {T} K {K} N {N} {dt}")
    dtype = DT[dt]
    x, w, bias = big(1, T, K, dtype=dtype), big(2, N, K, std=K ** -.5, dtype=dtype), big(3, N, dtype=dtype)
    for act in ("none", "gelu"):
        layer = Linear(w, bias, act=act)
        y, z = layer.forward(x, save=True)
        R.check("y", y, R.linear_forward(x.double(), w.double(), bias.double(), act, None, dtype, dtype)["y"])
        dout = big(4, T, N, std=.1, dtype=dtype)
        outs = layer.backward(x, dout, z, w_grad_dtype=torch.float32)
        ref = R.linear_backward(x.double(), w.double(), z.double(), dout.double(), act, dtype, dtype, torch.float32)
        for name, got in zip(("dx", "dw", "dbias"), outs):
            R.check(name, got, ref[name])
    wu = big(5, N, K, std=K ** -.5, dtype=dtype)
    gp = GatedProjection(w, wu, bias, bias)
    h, a, b = gp.forward(x, save=True)
    R.check("h", h, R.gated_forward(x.double(), w.double(), wu.double(), bias.double(), bias.double(), "silu", dtype)["h"])
    outs = gp.backward(x, a, b, dout, w_grad_dtype=torch.float32)
    ref = R.gated_backward(*(t.double() for t in (x, w, wu, a, b, dout)), "silu", dtype, torch.float32)
    for name, got in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), outs):
        R.check(name, got, ref[name])
