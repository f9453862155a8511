"""GPU tests of low-rank adapters of many requests against the 64-bit reference of tokens_ref.py:
types, ranks, odd sizes, strides, tokens without an adapter, adapters without a token, gradients,
graphs; and the whole way through norm, experts and adapters and back."""
import pytest
import torch

import dense_ref as R
import expert_cache_ffn_amd as ecf
import tokens_ref as TR
from expert_cache_ffn_amd.layer import GatedProjection, Linear, LowRankAdapters, RMSNorm, TokenSort
from gpu_util import say
from tokens_ref import DT, rand, strided

pytestmark = pytest.mark.gpu


def make(T, K, N, r, n, dt, od, seed=0, none=0.15):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, n, (T,), generator=g)
    ids = torch.where(torch.rand(T, generator=g) < none, torch.randint(-2, 0, (T,), generator=g) * 1000, ids)
    dtype, ot = DT[dt], DT[od]
    return dict(ids=ids.to(torch.int32).cuda(), x=rand(seed + 1, T, K, dtype=dtype), down=rand(seed + 2, n, r, K, std=K ** -.5, dtype=dtype),
                up=rand(seed + 3, n, N, r, std=r ** -.5, dtype=dtype), scale=(rand(seed + 4, n).abs() + 0.5),
                residual=rand(seed + 5, T, N, dtype=ot), dout=rand(seed + 6, T, N, std=0.1, dtype=ot), res_x=rand(seed + 7, T, K, std=0.1, dtype=dtype))


# (tokens, K, N, rank, adapters): single tokens and elements, both sides of the few tokens (in one launch and in two), ranks off the MFMA's 16 and
# over 64, many adapters of few tokens, one adapter of many, widths around every slice and chunk
SIZES = [(1, 1, 1, 1, 1), (1, 4096, 4096, 16, 64), (3, 7, 5, 3, 2), (16, 1000, 130, 16, 64), (64, 256, 264, 8, 3), (65, 64, 64, 4, 2),
         (66, 130, 257, 16, 40), (128, 128, 256, 32, 1), (200, 136, 72, 33, 5), (300, 520, 1030, 64, 4), (257, 1330, 300, 12, 1024),
         (700, 264, 136, 1, 9), (129, 300, 265, 100, 3), (90, 64, 72, 256, 2), (1500, 513, 384, 20, 7), (2100, 1024, 640, 16, 3),
         (5000, 8, 16, 5, 100), (40, 8200, 70, 12, 3), (64, 64, 5000, 8, 2), (7, 120, 1100, 2, 4), (9, 2000, 40, 6, 2)]
# enough tiles and columns for the waves of a block to take columns of their own, forward and backward
LARGE = [(700, 72, 12100, 12, 3), (700, 12100, 72, 20, 3), (650, 72, 12104, 48, 2), (650, 12104, 72, 64, 2)]
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T,K,N,r,n", SIZES + LARGE)
def test_forward(T, K, N, r, n, dt, od):
    say(f"case: adapters forward T {T} K {K} N {N} r {r} n {n} {dt} out {od}")
    q = make(T, K, N, r, n, dt, od)
    layer = LowRankAdapters(q["down"], q["up"], q["scale"], out_dtype=DT[od])
    ref = TR.adapters_forward(q, DT[dt], DT[od])
    y, h = layer.forward(q["x"], q["ids"], residual=q["residual"], save=True)
    R.check("h", h, ref["h"])
    R.check("out", y, ref["out"])
    s = TokenSort(q["ids"].long(), n)
    assert torch.equal(layer.forward(q["x"], s, residual=q["residual"]), y)
    kept = q["residual"].clone()
    assert layer.forward(q["x"], s, residual=kept, out=kept) is kept and torch.equal(kept, y)
    bare = LowRankAdapters(q["down"], q["up"], out_dtype=DT[od])
    q["residual"], q["scale"] = None, torch.ones(n, device="cuda")
    R.check("out", bare.forward(q["x"], q["ids"].long()), TR.adapters_forward(q, DT[dt], DT[od])["out"])


@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T,K,N,r,n", SIZES + LARGE)
def test_backward(T, K, N, r, n, dt, od):
    say(f"case: adapters backward T {T} K {K} N {N} r {r} n {n} {dt} out {od}")
    q = make(T, K, N, r, n, dt, od, seed=50)
    gd = torch.float32 if T % 2 else DT[dt]
    layer = LowRankAdapters(q["down"], q["up"], q["scale"], out_dtype=DT[od])
    q["h"] = TR.adapters_forward(q, DT[dt], DT[od])["h"][0].float()
    ref = TR.adapters_backward(q, DT[dt], gd)
    outs = layer.backward(q["x"], q["ids"], q["h"], q["dout"], residual=q["res_x"], w_grad_dtype=gd)
    for name, got in zip(("dx", "ddown", "dup"), outs):
        R.check(name, got, ref[name])
    s = TokenSort(q["ids"], n)
    for p, v in zip(layer.backward(q["x"], s, q["h"], q["dout"], residual=q["res_x"], w_grad_dtype=gd), outs):
        assert torch.equal(p, v), "two calls differ"
    kept = q["res_x"].clone()
    dx, none, none2 = layer.backward(q["x"], s, None, q["dout"], residual=kept, dx=kept, need_dw=False)
    assert dx is kept and none is none2 is None and torch.equal(dx, outs[0])
    none, *dw = layer.backward(q["x"], s, q["h"], q["dout"], w_grad_dtype=gd, need_dx=False)
    assert none is None and all(torch.equal(p, v) for p, v in zip(dw, outs[1:]))
    q["res_x"] = None
    R.check("dx", layer.backward(q["x"], s, q["h"], q["dout"], need_dw=False)[0], TR.adapters_backward(q, DT[dt], gd)["dx"])


@pytest.mark.parametrize("T", [5, 64, 65, 400])
def test_no_adapter_at_all_and_one_of_many(T):
    q = make(T, 72, 40, 8, 6, "bf16", "f32")
    layer = LowRankAdapters(q["down"], q["up"], q["scale"], out_dtype=torch.float32)
    for ids in (torch.full((T,), -1), torch.full((T,), 6)):
        y, h = layer.forward(q["x"], ids.cuda(), residual=q["residual"], save=True)
        assert torch.equal(y, q["residual"]) and not h.any()
        assert not layer.forward(q["x"], ids.cuda()).any()
        dx, ddown, dup = layer.backward(q["x"], ids.cuda(), h, q["dout"], residual=q["res_x"])
        assert torch.equal(dx, q["res_x"]) and not ddown.any() and not dup.any()
    q["ids"] = torch.full((T,), 4, dtype=torch.int32).cuda()
    ref = TR.adapters_forward(q, torch.bfloat16, torch.float32)
    y, q["h"] = layer.forward(q["x"], q["ids"], residual=q["residual"], save=True)
    R.check("out", y, ref["out"])
    back = TR.adapters_backward(q, torch.bfloat16, torch.bfloat16)
    for name, got in zip(("dx", "ddown", "dup"), layer.backward(q["x"], q["ids"], q["h"], q["dout"], residual=q["res_x"])):
        R.check(name, got, back[name])
        if name != "dx":
            assert not got[:4].any() and not got[5:].any()


def test_no_tokens():
    q = make(0, 16, 24, 4, 3, "f32", "f32")
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    y, h = layer.forward(q["x"], q["ids"], save=True)
    assert y.shape == (0, 24) and h.shape == (0, 4)
    dx, ddown, dup = layer.backward(q["x"], q["ids"], h, q["dout"])
    assert dx.shape == (0, 16) and not ddown.any() and not dup.any()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T", [10, 150])
def test_strides(T, dt):
    K, N, r, n, pad = 101, 203, 9, 4, 5
    q = make(T, K, N, r, n, dt, dt)
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    want, h = layer.forward(q["x"], q["ids"], residual=q["residual"], save=True)
    out, buf = strided(torch.zeros_like(want), pad, 3)
    got = layer.forward(strided(q["x"], 3, 1)[0], q["ids"], residual=strided(q["residual"], 1, 1)[0], out=out)
    assert torch.equal(got, want) and torch.isnan(buf[:3]).all() and torch.isnan(buf[3:].view(T, N + pad)[:, N:]).all()
    dx, buf = strided(torch.zeros_like(q["x"]), pad, 1)
    want_b = layer.backward(q["x"], q["ids"], h, q["dout"], residual=q["res_x"])
    got_b = layer.backward(strided(q["x"], 3, 1)[0], q["ids"], h, strided(q["dout"], 7, 5)[0], residual=strided(q["res_x"], 2, 3)[0], dx=dx)
    for p, v in zip(got_b, want_b):
        assert torch.equal(p, v)
    assert torch.isnan(buf[1:].view(T, K + pad)[:, K:]).all()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T", [12, 140])
def test_infinities_stay_in_their_rows(T, dt):
    """A token's infinities and NaN reach its own outputs, its adapter's gradients and no others'."""
    q = make(T, 96, 80, 8, 3, dt, dt, none=0)
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    clean, h = layer.forward(q["x"], q["ids"], save=True)
    dx0, dd0, du0 = layer.backward(q["x"], q["ids"], h, q["dout"])
    x, dout, hb = q["x"].clone(), q["dout"].clone(), h.clone()
    x[7, 3], dout[7, 5], hb[7, 2] = float("inf"), float("nan"), float("inf")
    out, _ = layer.forward(x, q["ids"], save=True)
    dx, dd, du = layer.backward(x, q["ids"], hb, dout)
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(out[keep], clean[keep]) and torch.equal(dx[keep], dx0[keep])
    others = torch.arange(3, device="cuda") != int(q["ids"][7])
    assert torch.equal(dd[others], dd0[others]) and torch.equal(du[others], du0[others])


@pytest.mark.parametrize("T", [10, 100])
def test_fp16_subnormals(T):
    """Adapters of fp16's smallest numbers, as they are early in training, keep their products."""
    K, N, r, n = 256, 64, 16, 2
    q = make(T, K, N, r, n, "f16", "f16", none=0)
    q["down"], q["up"] = rand(1, n, r, K, std=1e-6).half(), rand(2, n, N, r, std=1e-6).half()
    q["dout"], q["res_x"] = rand(3, T, N, std=1e-6).half(), None
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    _, q["h"] = layer.forward(q["x"], q["ids"], save=True)
    R.check("h", q["h"], TR.adapters_forward(q, torch.float16, torch.float16)["h"])
    q["h"] = q["h"] * 1e3
    back = TR.adapters_backward(q, torch.float16, torch.float32)
    _, dd, du = layer.backward(q["x"], q["ids"], q["h"], q["dout"], w_grad_dtype=torch.float32)
    R.check("ddown", dd, back["ddown"])
    R.check("dup", du, back["dup"])


def test_gradient_against_differences():
    q = make(90, 40, 50, 6, 3, "f32", "f32")
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    _, h = layer.forward(q["x"], q["ids"], save=True)
    grads = layer.backward(q["x"], q["ids"], h, q["dout"])
    names, e = ("x", "down", "up"), 1e-4

    def loss(p):
        f = {k: v.double() for k, v in q.items() if v.is_floating_point()} | p
        total = 0
        for i in range(3):
            at = (q["ids"] == i).nonzero().view(-1)
            total = total + (f["scale"][i] * (f["x"][at] @ f["down"][i].t() @ f["up"][i].t()) * f["dout"][at]).sum()
        return total

    for name, g in zip(names, grads):
        step = rand(9, *g.shape).double()
        slope = (loss({name: q[name].double() + e * step}) - loss({name: q[name].double() - e * step})) / (2 * e)
        assert abs(float((g.double() * step).sum() - slope)) <= 1e-5 * float((g.double() * step).abs().sum())


@pytest.mark.parametrize("T", [20, 300])
def test_graph(T):
    q = make(T, 264, 520, 16, 5, "bf16", "bf16")
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])

    def step():
        y, h = layer.forward(q["x"], q["ids"], residual=q["residual"], save=True)
        return [y, h, *layer.backward(q["x"], q["ids"], h, q["dout"])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = step()
    torch.cuda.synchronize()
    for seed in range(4):
        new = make(T, 264, 520, 16, 5, "bf16", "bf16", seed=100 * seed)
        q["x"].copy_(new["x"])
        q["ids"].copy_(new["ids"])
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, v in zip(kept, want):
            assert torch.equal(p, v)


def test_long_offsets():
    """Outputs and tokens past 2^31 elements."""
    T, K, N, r, n = 70000, 64, 32000, 8, 3
    q = make(T, K, 8, r, n, "bf16", "bf16")
    up = rand(3, n, N, r, std=r ** -.5, dtype=torch.bfloat16)
    layer = LowRankAdapters(q["down"], up, q["scale"])
    y, h = layer.forward(q["x"], q["ids"], save=True)
    assert y.numel() > 1 << 31
    tail = {"x": q["x"][-40:], "ids": q["ids"][-40:], "down": q["down"], "up": up, "scale": q["scale"], "residual": None}
    R.check("out", y[-40:], TR.adapters_forward(tail, torch.bfloat16, torch.bfloat16)["out"])
    dx, _, _ = layer.backward(q["x"], q["ids"], h, y, need_dw=False)
    tail |= {"dout": y[-40:], "h": h[-40:], "res_x": None}
    R.check("dx", dx[-40:], TR.adapters_backward(tail, torch.bfloat16, torch.bfloat16)["dx"])


def test_refusals():
    q = make(70, 16, 24, 4, 3, "f32", "f32")
    layer = LowRankAdapters(q["down"], q["up"], q["scale"])
    x, ids = q["x"], q["ids"]
    h = torch.zeros(70, 4, device="cuda")
    bad = [lambda: LowRankAdapters(q["down"][0], q["up"]), lambda: LowRankAdapters(q["down"], q["up"][:2]),
           lambda: LowRankAdapters(q["down"], q["up"].bfloat16()), lambda: LowRankAdapters(q["down"][:, :, ::2], q["up"]),
           lambda: LowRankAdapters(q["down"], q["up"], q["scale"].double()),
           lambda: LowRankAdapters(q["down"], q["up"], out_dtype=torch.float16), lambda: layer.forward(x, ids[:69]),
           lambda: layer.forward(x, ids.float()), lambda: layer.forward(x, None), lambda: layer.forward(x, TokenSort(ids, 4)),
           lambda: layer.forward(x, TokenSort(ids[:69], 3)), lambda: layer.forward(x[:, :8], ids),
           lambda: layer.forward(x, ids, residual=q["residual"][:, :8]), lambda: layer.backward(x, ids, h[:, :3], q["dout"]),
           lambda: layer.backward(x, ids, None, q["dout"]), lambda: layer.backward(x, ids, h, q["dout"], need_dx=False, dx=x)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    with pytest.raises(ecf.EcfError):
        LowRankAdapters(torch.zeros(1, 300, 8, device="cuda"), torch.zeros(1, 8, 300, device="cuda"))
    with pytest.raises(ecf.EcfError):  # dx onto x
        layer.backward(x, ids, h, q["dout"], dx=x)


def test_a_layer_of_all_of_them():
    """norm -> sort -> experts whose first product has adapters -> combine onto the running sum, and back, in fp32
    against torch's gradients in 64 bits."""
    T, d, I, E, k, r, n = 150, 128, 96, 5, 2, 8, 3
    p = {"weight": 1 + rand(1, d, std=0.1), "up": rand(2, E, I, d, std=d ** -.5), "out": rand(3, E, d, I, std=I ** -.5),
         "a": rand(4, n, r, d, std=d ** -.5), "b": rand(5, n, I, r, std=r ** -.5), "x": rand(6, T, d), "residual": rand(7, T, d)}
    scale = rand(8, n).abs() + 0.5
    g = torch.Generator().manual_seed(9)
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    ids[140:] = -1  # padding
    request = torch.randint(-1, n, (T,), generator=g).to(torch.int32)
    gates = rand(10, T, k).softmax(1)
    dout = rand(11, T, d, std=0.1)
    ids, request = ids.cuda(), request.cuda()

    def ours():
        norm = RMSNorm(p["weight"])
        o = norm.forward(p["x"], residual=p["residual"], save=True)
        s = TokenSort(ids, E)
        rows = s.dispatch(o.y)
        of_rows = torch.where(s.order < 140 * k, request[s.order.long() // k], -1)  # each row's request
        adapters = LowRankAdapters(p["a"], p["b"], scale)
        by = TokenSort(of_rows, n)
        at = s.offsets.tolist()
        z = torch.zeros(T * k, I, device="cuda")
        for e in range(E):
            if at[e + 1] > at[e]:
                Linear(p["up"][e]).forward(rows[at[e]:at[e + 1]], out=z[at[e]:at[e + 1]])
        z, h = adapters.forward(rows, by, residual=z, save=True)
        y = torch.zeros(T * k, d, device="cuda")
        for e in range(E):
            if at[e + 1] > at[e]:
                Linear(p["out"][e]).forward(torch.relu(z[at[e]:at[e + 1]]), out=y[at[e]:at[e + 1]])
        out = s.combine(y, gates, residual=o.sum)
        dy, dgates = s.combine_backward(y, gates, dout)
        grads = {"up": torch.zeros_like(p["up"]), "out": torch.zeros_like(p["out"])}
        dz, drows = torch.zeros_like(z), torch.zeros_like(rows)
        for e in range(E):
            q = slice(at[e], at[e + 1])
            if at[e + 1] > at[e]:
                dact, grads["out"][e], _ = Linear(p["out"][e]).backward(torch.relu(z[q]), dy[q])
                dz[q] = dact * (z[q] > 0)
                drows[q], grads["up"][e], _ = Linear(p["up"][e]).backward(rows[q], dz[q])
        drows, grads["a"], grads["b"] = adapters.backward(rows, by, h, dz, residual=drows)
        dnorm = s.dispatch_backward(drows)
        grads["x"], grads["residual"], grads["weight"] = norm.backward(o.sum, o.rstd, dnorm, dsum=dout)
        return out, dgates, grads

    out, dgates, grads = ours()
    f = {name: v.double().requires_grad_() for name, v in p.items()}
    w = gates.double().requires_grad_()
    total = f["x"] + f["residual"]
    y = total / torch.sqrt((total * total).mean(1, keepdim=True) + 1e-6) * f["weight"]
    back = 0
    for j in range(k):
        e, live = ids[:, j].long().clamp_min(0), (ids[:, j] >= 0)[:, None]
        z = (f["up"][e] * y[:, None]).sum(2)
        a, on = request.long().clamp_min(0), (request >= 0)[:, None]
        low = (f["a"][a] * y[:, None]).sum(2) * scale.double()[a][:, None]
        z = z + on * (f["b"][a] * low[:, None]).sum(2)
        back = back + live * w[:, j:j + 1] * (f["out"][e] * torch.relu(z)[:, None]).sum(2)
    want = total + back
    want.backward(dout.double())
    # chains of fp32 products and sums: a hundred steps of 2^-23 each, relative to the tensor's size
    for name, got, ref in [("out", out, want.detach()), ("gates", dgates, w.grad)] + [(m, grads[m], f[m].grad) for m in grads]:
        assert (got.double() - ref).abs().max() <= 100 * TR.E23 * ref.abs().max(), name


def test_8_bit_tokens_through_gated_experts():
    """norm -> 8 bits -> sort -> gated experts -> combine, as a decode batch would, against the same from the values that the
    8 bits stand for."""
    T, d, I, E, k = 24, 256, 128, 6, 2
    norm = RMSNorm(1 + rand(1, d, std=0.1, dtype=torch.bfloat16).float().to(torch.bfloat16), sum_dtype=torch.float32)
    x, res = rand(2, T, d, dtype=torch.bfloat16), rand(3, T, d)
    o = norm.forward(x, residual=res, mx=True, y=False)
    ids = torch.rand(T, E, generator=torch.Generator().manual_seed(4)).topk(k, dim=1).indices.cuda()
    s, gates = TokenSort(ids, E), rand(5, T, k).softmax(1)
    rows = s.dispatch(o.q, scale=o.scale, dtype=torch.bfloat16)
    assert torch.equal(rows, TR.mx_values(o.q, o.scale).to(torch.bfloat16)[s.order.long() // k])
    wg, wu, wd = (rand(6 + i, E, *sh, std=sh[1] ** -.5, dtype=torch.bfloat16) for i, sh in enumerate([(I, d), (I, d), (d, I)]))
    y, at = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda"), s.offsets.tolist()
    for e in range(E):
        if at[e + 1] > at[e]:
            h = GatedProjection(wg[e], wu[e]).forward(rows[at[e]:at[e + 1]])
            Linear(wd[e]).forward(h, out=y[at[e]:at[e + 1]])
    out = s.combine(y, gates, residual=o.sum)
    R.check("out", out, TR.combine(y, s.place, T * k, gates, o.sum, torch.float32))
