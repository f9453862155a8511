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
