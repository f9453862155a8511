"""GPU tests of the token operators at the largest documented numbers of tokens and choices."""
import pytest
import torch

import dense_ref as R
import tokens_ref as TR
from expert_cache_ffn_amd.layer import RMSNorm, TokenSort
from gpu_util import say
from tokens_ref import rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def needs(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of free GPU memory")


def test_norm_of_the_most_tokens():
    """2^22 rows over 8192 elements: a block of 1024 threads each."""
    needs(130)
    T, d, period = 1 << 22, 8200, 1024
    say(f"case: norm T {T} d {d} bf16 to 8 bits")
    base = rand(1, period, d, dtype=torch.bfloat16)
    x = base.repeat(T // period, 1)
    own = [slice(0, 40), slice((1 << 21) - 40, (1 << 21) + 40), slice(T - 40, T)]
    for i, s in enumerate(own):
        x[s] = rand(10 + i, s.stop - s.start, d, std=1.0 + i, dtype=torch.bfloat16)
    norm = RMSNorm(1 + rand(2, d, std=0.1, dtype=torch.bfloat16))
    o = norm.forward(x, y=False, mx=True, save=True)
    assert o.q.numel() > 1 << 34
    want = norm.forward(base, y=False, mx=True, save=True)
    for s in own:
        part = norm.forward(x[s], y=False, mx=True, save=True)
        for name in ("q", "scale", "rstd"):
            a, b = getattr(o, name)[s], getattr(part, name)
            assert torch.equal(a.view(torch.uint8) if name != "rstd" else a, b.view(torch.uint8) if name != "rstd" else b), name
            getattr(o, name)[s] = getattr(want, name)[torch.arange(s.start, s.stop, device="cuda") % period]
    for name in ("q", "scale", "rstd"):
        a, b = getattr(o, name), getattr(want, name)
        if name != "rstd":
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        for t in range(0, T, period * 64):
            assert (a[t:t + period * 64].view(64, period, -1) == b.view(1, period, -1)).all(), (name, t)


def test_combine_backward_of_the_most_choices():
    """2^26 choices of rows over 256 elements: a wave each."""
    needs(100)
    T, k, E, d = 1 << 21, 32, 7, 264
    say(f"case: combine backward T {T} k {k} E {E} d {d} bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    s = TokenSort(ids, E)
    live = int(s.offsets[-1])
    assert live == int((ids >= 0).sum()) and s.counts.tolist() == [int((ids == e).sum()) for e in range(E)]
    rows = torch.randn(1 << 20, d, generator=g, device="cuda").to(torch.bfloat16).repeat(64, 1)
    gates = torch.rand(T, k, generator=g, device="cuda")
    dout = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    drows, dgates = s.combine_backward(rows, gates, dout)
    assert not drows[live:].any()
    for t in (slice(0, 20), slice(T // 2 - 10, T // 2 + 10), slice(T - 20, T)):
        at, ok = s.place[t].long(), s.place[t] < live
        assert torch.equal(at < live, ids[t] >= 0)
        terms = torch.where(ok[:, :, None], rows[at].double() * dout[t].double()[:, None], 0.0)
        R.check("dgates", dgates[t], (terms.sum(2), terms.abs().sum(2) * 12 * TR.E23 + 1e-37))
        want = torch.where(ok, gates[t], 0.0)[:, :, None] * dout[t].float()[:, None]
        assert torch.equal(drows[at], want.to(torch.bfloat16))
