"""GPU tests of how many bits the low-rank adapters keep between their products.  The inputs are such that
every product and every partial sum, in any order, is exact in fp32, and the large parts of the rank-wide values
cancel: what is left is their last 8 of 24 bits, and outputs have to be equal to the bit."""
import pytest
import torch

from expert_cache_ffn_amd.layer import LowRankAdapters
from gpu_util import say
from tokens_ref import DT

pytestmark = pytest.mark.gpu

PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def pieces(g, n):
    """[n, 3]: three numbers of 8 bits whose sum u in [1, 1.75) has 24 (each a multiple of 2^-23)."""
    hi, mid, lo = (torch.randint(a, b, (n,), generator=g, dtype=torch.float64) for a, b in ((128, 224), (1, 256), (0, 128)))
    return torch.stack([hi * 2.0 ** -7, mid * 2.0 ** -15, (2 * lo + 1) * 2.0 ** -23], 1)


def powers(g, *shape):
    return 2.0 ** torch.randint(-1, 3, shape, generator=g).double()


def equal(name, got, want):
    """want is in 64 bits, and of got's type without rounding."""
    assert torch.equal(want.to(got.dtype).double(), want), f"{name}: the case is not exact"
    off = (got.double() - want).abs().max()
    assert torch.equal(got.double(), want), f"{name}: off by {float(off)} of {float(want.abs().max())}"


def case(seed, T, K, N, r, n):
    """Zeros: ids, scale (powers of two), x, down, up, in 64 bits on the CPU."""
    g = torch.Generator().manual_seed(seed)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    return g, dict(ids=torch.randint(0, n, (T,), generator=g), scale=powers(g, n).clamp(1, 2), x=z(T, K), down=z(n, r, K), up=z(n, N, r),
                   dout=z(T, N))


def layer_of(q, dt, od):
    return LowRankAdapters(q["down"].to(DT[dt]).cuda(), q["up"].to(DT[dt]).cuda(), q["scale"].float().cuda(), out_dtype=DT[od])


# (tokens, widths, rank): a few tokens in one launch and in two; slices of 128 columns and of 512; one, two and more steps of ranks
FORWARD = [(20, 300, 72, 2), (20, 300, 72, 100), (20, 9000, 72, 16), (150, 300, 72, 2), (150, 300, 200, 8), (150, 520, 72, 16),
           (150, 300, 72, 20), (150, 2100, 72, 32), (150, 300, 72, 33), (150, 300, 130, 64), (150, 300, 72, 100), (90, 64, 72, 256),
           (700, 72, 12100, 12), (700, 72, 12100, 30), (700, 72, 12100, 48)]


@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T,K,N,r", FORWARD)
def test_forward_keeps_24_bits(T, K, N, r, dt, od):
    say(f"case: exact forward T {T} K {K} N {N} r {r} {dt} out {od}")
    n = 3
    g, q = case(T + r, T, K, N, r, n)
    at = [0, K // 2, K - 1]
    q["x"][:, at] = p = pieces(g, T)
    q["down"][:, r - 1, at] = 1
    q["down"][:, 0, at[:2]] = -1  # h[0] + h[r - 1] is the third piece
    c = powers(g, n, N)
    q["up"][:, :, 0] = q["up"][:, :, r - 1] = c
    ids = q["ids"].int().cuda()
    out, h = layer_of(q, dt, od).forward(q["x"].to(DT[dt]).cuda(), ids, save=True)
    equal("h", h[:, r - 1].cpu(), p.sum(1))
    equal("out", out.cpu(), (q["scale"][:, None] * c)[q["ids"]] * p[:, 2:])
    if od == "f32":  # all of it
        q["up"][:, :, 0] = 0
        equal("out", layer_of(q, dt, od).forward(q["x"].to(DT[dt]).cuda(), ids).cpu(),
              (q["scale"][:, None] * c)[q["ids"]] * p.sum(1, keepdim=True))


@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T,N,K,r", [s for s in FORWARD if s[0] > 64] + [(20, 300, 72, 16)])
def test_dx_keeps_24_bits(T, K, N, r, dt, od):
    say(f"case: exact dx T {T} K {K} N {N} r {r} {dt} out {od}")
    n = 3
    g, q = case(T + r, T, K, N, r, n)
    at = [0, N // 2, N - 1]
    q["dout"][:, at] = p = pieces(g, T)
    q["up"][:, at, r - 1] = 1
    q["up"][:, at[:2], 0] = -1
    c = powers(g, n, K)
    q["down"][:, 0] = q["down"][:, r - 1] = c
    ids, x = q["ids"].int().cuda(), q["x"].to(DT[dt]).cuda()
    want = (q["scale"][:, None] * c)[q["ids"]] * p[:, 2:]
    dx, _, _ = layer_of(q, dt, od).backward(x, ids, None, q["dout"].to(DT[od]).cuda(), need_dw=False)
    equal("dx", dx.cpu(), want)
    if od == "f32":  # dout itself has 24 bits, and the sum over its columns cancels
        q["dout"].zero_()
        q["dout"][:, at[0]], q["dout"][:, at[2]] = p.sum(1), -p[:, :2].sum(1)
        q["up"].zero_()
        q["up"][:, :, r - 1] = 1
        dx, _, _ = layer_of(q, dt, od).backward(x, ids, None, q["dout"].to(DT[od]).cuda(), need_dw=False)
        equal("dx", dx.cpu(), want)


@pytest.mark.parametrize("gd", ["same", "f32"])
@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T,K,N,r,n", [(200, 136, 72, 2, 100), (200, 72, 136, 16, 100), (200, 72, 72, 20, 100), (200, 72, 72, 33, 100),
                                       (200, 300, 72, 64, 100), (200, 72, 72, 100, 100), (1500, 72, 300, 8, 1), (1500, 300, 72, 40, 1)])
def test_weight_gradients_keep_24_bits(T, K, N, r, n, dt, od, gd):
    """Two tokens of each adapter have something; of the only one, in different runs of the order."""
    say(f"case: exact gradients T {T} K {K} N {N} r {r} n {n} {dt} out {od} gradients {gd}")
    g, q = case(T + r, T, K, N, r, n)
    q["ids"] = torch.arange(T) % n
    first, second = torch.arange(n), torch.arange(T - n, T) if n > 1 else torch.tensor([T - 3])
    p, j, at = pieces(g, n), r - 1, [0, N // 2, N - 1]
    gt = torch.float32 if gd == "f32" else DT[dt]
    # ddown: g of the first token is u, that of the second takes the first two pieces off again
    for k in range(3):
        q["dout"][first, at[k]] = p[:, k]
        if k < 2:
            q["dout"][second, at[k]] = -p[:, k]
    q["up"][:, at, j] = 1
    c = powers(g, n, K)
    q["x"][first] = q["x"][second] = c
    ids, x = q["ids"].int().cuda(), q["x"].to(DT[dt]).cuda()
    h = torch.zeros(T, r, dtype=torch.float64)
    _, ddown, _ = layer_of(q, dt, od).backward(x, ids, h.float().cuda(), q["dout"].to(DT[od]).cuda(), w_grad_dtype=gt, need_dx=False)
    want = torch.zeros(n, r, K, dtype=torch.float64)
    want[:, j] = q["scale"][:, None] * p[:, 2:] * c
    equal("ddown", ddown.cpu(), want)
    # dup: the same of h
    h[first, j], h[second, j] = p.sum(1), -p[:, :2].sum(1)
    c = powers(g, n, N)
    q["dout"].zero_()
    q["dout"][first] = q["dout"][second] = c
    _, _, dup = layer_of(q, dt, od).backward(x, ids, h.float().cuda(), q["dout"].to(DT[od]).cuda(), w_grad_dtype=gt, need_dx=False)
    want = torch.zeros(n, N, r, dtype=torch.float64)
    want[:, :, j] = q["scale"][:, None] * c * p[:, 2:]
    equal("dup", dup.cpu(), want)


def same(name, got, want):
    assert torch.equal(got.double().cpu(), want.to(got.dtype).double()), f"{name}: {got.flatten()[:4]} for {want.flatten()[:4]}"


@pytest.mark.parametrize("dt,od", [p for p in PAIRS if p[0] != "f16"])
@pytest.mark.parametrize("T", [20, 150])
def test_the_largest_finite_values(T, dt, od):
    """h, g and dout next to the largest fp32 number, which a bf16 number rounds to infinity, times small ones."""
    K, N, r, n, small = 64, 72, 8, 2, 2.0 ** -100
    big = (2 - 2.0 ** -7) * 2.0 ** 127 + 1.5 * 2.0 ** 119  # over the middle between bf16's largest number and 2^128
    pair = torch.tensor([(2 - 2.0 ** -7) * 2.0 ** 63, 1.5 * 2.0 ** 55], dtype=torch.float64)
    _, q = case(T, T, K, N, r, n)
    q["x"][7, :2], q["down"][:, 5, :2], q["up"][:, :, 5] = pair, 2.0 ** 64, small
    q["scale"].fill_(1)
    ids, none = q["ids"].int().cuda(), torch.zeros(T, r, device="cuda")
    out, h = layer_of(q, dt, od).forward(q["x"].to(DT[dt]).cuda(), ids, save=True)
    want = torch.zeros(T, r, dtype=torch.float64)
    want[7, 5] = big
    same("h", h, want)
    same("out", out, (big * small * (torch.arange(T) == 7))[:, None].expand(T, N).double())
    # the same through g, from a product or (dout in fp32) from one value
    _, q = case(T, T, K, N, r, n)
    q["scale"].fill_(1)
    a = int(q["ids"][7])
    douts = [(pair, 2.0 ** 64)] + ([(torch.tensor([big, 0.0]), 1.0)] if od == "f32" else [])
    for values, up in douts:
        q["dout"][7, :2], q["up"][:, :2, 5], q["down"][:, 5] = values.double(), up, small
        q["x"][7] = small
        dx, ddown, _ = layer_of(q, dt, od).backward(q["x"].to(DT[dt]).cuda(), ids, none, q["dout"].to(DT[od]).cuda())
        same("dx", dx, (big * small * (torch.arange(T) == 7))[:, None].expand(T, K).double())
        want = torch.zeros(n, r, K, dtype=torch.float64)
        want[a, 5] = big * small
        same("ddown", ddown, want)
    h = none.clone()
    h[7, 5] = big
    q["dout"].zero_()
    q["dout"][7] = small
    _, _, dup = layer_of(q, dt, od).backward(q["x"].to(DT[dt]).cuda(), ids, h, q["dout"].to(DT[od]).cuda())
    want = torch.zeros(n, N, r, dtype=torch.float64)
    want[a, :, 5] = big * small
    same("dup", dup, want)


@pytest.mark.parametrize("dt,od", PAIRS)
@pytest.mark.parametrize("T", [20, 150])
def test_infinities_stay_infinities(T, dt, od):
    """An infinite h, g or dout times numbers other than zero is one of their signs, as in the formulas; a NaN stays one."""
    K, N, r, n, inf = 64, 72, 8, 2, float("inf")
    g, q = case(T, T, K, N, r, n)
    q["down"], q["up"], q["x"] = powers(g, n, r, K), powers(g, n, N, r), powers(g, T, K)
    q["up"][:, ::2] *= -1
    q["down"][:, :, ::2] *= -1
    q["x"][:, ::2] *= -1
    q["dout"] = powers(g, T, N)
    q["dout"][:, ::2] *= -1
    x, dout, ids = q["x"].clone(), q["dout"].clone(), q["ids"].int().cuda()
    layer = layer_of(q, dt, od)
    a = int(q["ids"][7])
    x[7, 0], x[9, 3] = -inf, float("nan")
    out, h = layer.forward(x.to(DT[dt]).cuda(), ids, save=True)
    same("h", h[7], torch.full((r,), inf).double())
    same("out", out[7], inf * q["up"][a, :, 0])
    assert torch.isnan(out[9]).all() and torch.isfinite(out[10:]).all()
    dout[7, 0] = -inf  # g is +inf
    ones = torch.ones(T, r, device="cuda")
    dx, ddown, dup = layer.backward(q["x"].to(DT[dt]).cuda(), ids, ones, dout.to(DT[od]).cuda())
    same("dx", dx[7], inf * q["down"][a, 0])
    same("ddown", ddown[a], (inf * q["x"][7]).expand(r, K))
    if od == "bf16":  # an infinite operand meets all parts of h, zeros among them: infinite or NaN
        assert not torch.isfinite(dup[a, 0]).any()
    else:
        same("dup", dup[a, 0], torch.full((r,), -inf).double())
    assert torch.isfinite(dx[10:]).all() and torch.isfinite(ddown[1 - a]).all() and torch.isfinite(dup[:, 1:]).all()
    ones[7, 5] = -inf
    _, _, dup = layer.backward(q["x"].to(DT[dt]).cuda(), ids, ones, q["dout"].to(DT[od]).cuda())
    same("dup", dup[a, :, 5], -inf * q["dout"][7])
    dout[7, 0] = float("nan")
    dx, ddown, _ = layer.backward(q["x"].to(DT[dt]).cuda(), ids, torch.ones(T, r, device="cuda"), dout.to(DT[od]).cuda())
    assert torch.isnan(dx[7]).all() and torch.isnan(ddown[a]).all() and torch.isfinite(dx[10:]).all()
