"""GPU tests of the norm's 8-bit output next to the borders of its scales: a group whose largest value lies as near to
448 times a power of two as fp32 inputs allow has the least scale that holds it, by the definition in 64 bits."""
import pytest
import torch

import tokens_ref as TR
from expert_cache_ffn_amd.layer import RMSNorm
from gpu_util import say

pytestmark = pytest.mark.gpu

EPS = 1e-6


def exact(s, w):
    v = (s.double() ** 2).mean(1, keepdim=True) + float(torch.tensor(EPS, dtype=torch.float32))
    return s.double() / v.sqrt() * w.double()


def next_up(m, up):
    return torch.nextafter(m, torch.full_like(m, float("inf") if up else 0.0))


def borders(seed, T, d, at, e):
    """(sums in fp32, weights): in column `at` of rows 0, 2, .. the largest value with |y| <= 1.75 * 2^e, in the rows
    after them the next one; the group's other values are smaller."""
    g = torch.Generator().manual_seed(seed)
    w = (1 + 0.1 * torch.randn(d, generator=g)).float()
    s = torch.randn(T, d, generator=g).float()
    group = at // 32 * 32
    s[:, group:group + 32] *= 0.25
    s[1::2] = s[::2]
    rest = (s.double() ** 2).sum(1) - s[:, at].double() ** 2
    k = (1.75 * 2.0 ** e / w[at].double()) ** 2 / d  # m^2 = k (m^2 + rest + d eps)
    m = torch.sqrt(k * (rest + d * EPS) / (1 - k)).float()
    for _ in range(8):  # to the largest fp32 number within the border
        s[:, at] = m
        over = exact(s, w)[:, at].abs() > 1.75 * 2.0 ** e
        m = torch.where(over, next_up(m, False), m)
    for _ in range(8):
        s[:, at] = up = next_up(m, True)
        over = exact(s, w)[:, at].abs() > 1.75 * 2.0 ** e
        m = torch.where(over, m, up)
    s[:, at] = m
    s[1::2, at] = next_up(m, True)[1::2]
    s[:, at] *= torch.where(torch.rand(T, generator=g) < 0.5, -1.0, 1.0)
    return s, w


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,at,e", [(400, 96, 5, 0), (2000, 100, 98, 0), (2000, 999, 31, 1), (600, 4096, 4000, 1), (300, 5001, 7, 2),
                                      (60, 12000, 8200, 2), (40, 20004, 20003, 2), (40, 20000, 16384, 2)])
def test_scales_next_to_their_borders(T, d, at, e, dt):
    say(f"case: norm borders T {T} d {d} column {at} {dt}")
    s, w = borders(T + d, T, d, at, e)
    y = exact(s, w)
    low, high = y[::2, at].abs(), y[1::2, at].abs()
    near = 1.75 * 2.0 ** e
    assert (low <= near).all() and (high > near).all() and (high / low < 1 + 2.0 ** -21).all()
    assert (y[:, at].abs() >= y[:, at // 32 * 32:at // 32 * 32 + 32].abs().amax(1)).all()
    want = TR.mx_bytes(y)
    assert (want[1::2, at // 32] == want[::2, at // 32] + 1).all()
    s, w = s.cuda(), w.cuda()
    if dt == "f32":
        o = RMSNorm(w, eps=EPS).forward(s, mx=True)
    else:  # as a residual stream in fp32
        o = RMSNorm(w, eps=EPS, dtype=torch.bfloat16, sum_dtype=torch.float32).forward(torch.zeros_like(s, dtype=torch.bfloat16), residual=s, mx=True)
    b = o.scale.view(torch.uint8).long().cpu()
    wrong = int((b[:, at // 32] != want[:, at // 32]).sum())
    assert wrong == 0, f"{wrong} of {T} scales are not the least"
    q = o.q.float().cpu()
    assert torch.isfinite(q).all()
    top = q[:, at].abs()
    assert (top[::2] == 448).all() and (top[1::2] == 224).all()
    TR.check_mx(o.q, o.scale, (y.cuda(), 2 * TR.E23 * y.abs().cuda()))


def test_infinite_values_beside_a_border():
    """An infinite or NaN weight makes its own elements NaN, and has no part in the scale."""
    s, w = borders(3, 400, 96, 5, 0)
    for bad in (float("inf"), float("nan")):
        wb = w.clone()
        wb[9] = bad
        y = exact(s, wb)
        o = RMSNorm(wb.cuda(), eps=EPS).forward(s.cuda(), mx=True)
        assert torch.equal(o.scale.view(torch.uint8).long().cpu(), TR.mx_bytes(y).long())
        q = o.q.float().cpu()
        assert torch.isnan(q[:, 9]).all() and torch.isfinite(q[:, :9]).all() and torch.isfinite(q[:, 10:]).all()
