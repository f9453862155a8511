"""GPU tests of how the token operators' entry points are called."""
import pytest
import torch

from expert_cache_ffn_amd.layer import LowRankAdapters
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
