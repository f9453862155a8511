"""GPU tests of how the token operators' entry points are called."""
import pytest
import torch

from expert_cache_ffn_amd.layer import LowRankAdapters, TokenSort
from tokens_ref import rand

pytestmark = pytest.mark.gpu


def stack(n=3, r=4, K=16, N=24):
    return rand(1, n, r, K), rand(2, n, N, r)


def test_a_scale_that_learns_is_refused():
    """The adapters' scale is a constant: backward() has no gradient for it."""
    down, up = stack()
    scale = torch.ones(3, device="cuda", requires_grad=True)
    for mode in (torch.enable_grad, torch.no_grad):
        with mode(), pytest.raises(ValueError, match="constant"):
            LowRankAdapters(down, up, scale)
    x, ids = rand(3, 70, 16), torch.arange(70, dtype=torch.int32, device="cuda") % 3
    assert torch.equal(LowRankAdapters(down, up, scale.detach()).forward(x, ids), LowRankAdapters(down, up).forward(x, ids))


@pytest.mark.parametrize("T", [40, 130])
def test_adapters_take_any_sort(T):
    """A TokenSort over ids that do not lie one after the other (a column of a table), as one over their copy."""
    down, up = stack()
    table = torch.randint(-1, 3, (T, 5), generator=torch.Generator().manual_seed(T)).cuda()
    layer, x, dout = LowRankAdapters(down, up), rand(3, T, 16), rand(4, T, 24)
    flat = table[:, 2].contiguous()
    want, h = layer.forward(x, flat, save=True)
    grads = layer.backward(x, flat, h, dout)
    for ids in (table[:, 2], table[:, 2:3], table.int()[:, 2], flat[:, None]):
        s = TokenSort(ids, 3)
        out, low = layer.forward(x, s, save=True)
        assert torch.equal(out, want) and torch.equal(low, h)
        for p, q in zip(layer.backward(x, s, h, dout), grads):
            assert torch.equal(p, q)
