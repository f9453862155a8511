"""GPU tests of tokens sorted by expert and back, with gradients, against the references of
tokens_ref.py: the order exactly, types, odd sizes and strides, choices of no expert, offsets past
32 bits, graphs."""
import pytest
import torch

import dense_ref as R
import expert_cache_ffn_amd as ecf
import tokens_ref as TR
from expert_cache_ffn_amd.layer import RMSNorm, TokenSort
from gpu_util import say
from tokens_ref import DT, rand, strided

pytestmark = pytest.mark.gpu


def choices(seed, T, k, E, none=0.1, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    ids = (torch.randn(T, E, generator=g) + 2 * torch.randn(E, generator=g)).topk(min(k, E), dim=1).indices if E >= k \
        else torch.randint(0, E, (T, k), generator=g)
    drop = torch.rand(T, k, generator=g) < none
    ids = torch.where(drop, torch.randint(-3, 0, (T, k), generator=g), ids)
    ids = torch.where(drop & (torch.rand(T, k, generator=g) < 0.5), E + torch.randint(0, 5, (T, k), generator=g), ids)
    return ids.to(dtype).cuda()


def check_sort(s, ids, E):
    ref = TR.sort(ids, E)
    for name in ("counts", "offsets", "tiles", "order", "place"):
        got = getattr(s, name)
        assert got.dtype is torch.int32 and torch.equal(got.cpu().long(), ref[name]), name
    return int(ref["offsets"][-1])


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 256), (3, 2, 2), (5, 32, 40), (16, 6, 256), (63, 1, 7), (64, 1, 64), (65, 3, 5),
                                   (100, 8, 1024), (1024, 1, 1024), (1023, 4, 60), (1025, 1, 3), (1365, 3, 8), (2049, 2, 300),
                                   (4097, 1, 1), (4096, 6, 256), (8192, 8, 1023), (30000, 5, 33), (70001, 2, 17)])
def test_sort(T, k, E):
    for wide, none in ((torch.int32, 0.1), (torch.int64, 0.0)):
        say(f"case: sort T {T} k {k} E {E} {wide} none {none}")
        ids = choices(T + k, T, k, E, none, wide)
        check_sort(TokenSort(ids, E), ids, E)


@pytest.mark.parametrize("T,k,E", [(7, 3, 5), (3000, 2, 9)])
def test_sort_special(T, k, E):
    for ids in (torch.full((T, k), -1, dtype=torch.int32), torch.full((T, k), E, dtype=torch.int64),
                torch.full((T, k), E - 1, dtype=torch.int64), torch.full((T, k), (1 << 32) + 1, dtype=torch.int64),
                torch.full((T, k), -(1 << 31), dtype=torch.int32)):
        ids = ids.cuda()
        check_sort(TokenSort(ids, E), ids, E)
    wide = torch.randint(0, E, (T, k + 4), dtype=torch.int32).cuda()
    check_sort(TokenSort(wide[:, 2:2 + k], E), wide[:, 2:2 + k], E)
    flat = torch.randint(0, E, (T,), dtype=torch.int64).cuda()
    s = TokenSort(flat, E)
    assert s.place.shape == (T, 1)
    check_sort(s, flat, E)


def test_no_tokens():
    s = TokenSort(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4)
    assert s.counts.tolist() == [0] * 4 and s.offsets.tolist() == [0] * 5 and s.tiles.tolist() == [0] * 6
    x = torch.empty(0, 8, device="cuda")
    rows = s.dispatch(x)
    assert rows.shape == (0, 8) and s.combine(rows).shape == (0, 8)
    drows, dw = s.combine_backward(rows, torch.empty(0, 3, device="cuda"), x)
    assert drows.shape == (0, 8) and dw.shape == (0, 3)


# (tokens, k, experts, d)
SIZES = [(1, 1, 1, 1), (1, 6, 256, 4096), (2, 3, 4, 7), (5, 2, 3, 8), (16, 6, 256, 1000), (33, 4, 8, 65), (100, 8, 60, 129), (64, 9, 16, 264),
         (257, 32, 64, 40), (1000, 2, 5, 2731), (700, 5, 31, 512)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k,E,d", SIZES)
def test_moves(T, k, E, d, dt):
    say(f"case: moves T {T} k {k} E {E} d {d} {dt}")
    dtype = DT[dt]
    ids = choices(T + d, T, k, E)
    s = TokenSort(ids, E)
    live = check_sort(s, ids, E)
    place, order = s.place, s.order.long()
    x = rand(1, T, d, dtype=dtype)
    rows = s.dispatch(x)
    want = x[order // k].clone()
    want[live:] = 0
    assert torch.equal(rows, want)
    y = rand(2, T * k, d, dtype=dtype)
    y[live:] = float("nan")  # nobody's rows
    gates = rand(3, T, k).softmax(1)
    for od in {dtype, torch.float32}:
        res = rand(4, T, d, dtype=od)
        out = s.combine(y, gates, residual=res)
        assert out.dtype is od
        R.check("out", out, TR.combine(y, place, live, gates, res, od))
        kept = res.clone()
        assert s.combine(y, gates, residual=kept, out=kept) is kept and torch.equal(kept, out)
        R.check("out", s.combine(y, gates, out_dtype=od), TR.combine(y, place, live, gates, None, od))
        dout = rand(5, T, d, dtype=od)
        ref = TR.combine_backward(y, place, live, gates, dout, dtype)
        drows, dgates = s.combine_backward(y, gates, dout)
        R.check("drows", drows, ref["drows"])
        R.check("dweights", dgates, ref["dweights"])
        none, only = s.combine_backward(y, gates, dout, need_drows=False)
        assert none is None and torch.equal(only, dgates)
        only, none = s.combine_backward(y, gates, dout, need_dweights=False)
        assert none is None and torch.equal(only, drows)
    R.check("out", s.combine(y), TR.combine(y, place, live, None, None, dtype))
    R.check("drows", s.combine_backward(y, None, rand(5, T, d, dtype=dtype))[0],
            TR.combine_backward(y, place, live, None, rand(5, T, d, dtype=dtype), dtype)["drows"])
    dx = s.dispatch_backward(y, residual=x)
    R.check("dx", dx, TR.combine(y, place, live, None, x, dtype))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k,E,d", [(3, 2, 4, 7), (16, 6, 256, 4096), (100, 3, 5, 1000), (33, 1, 8, 40)])
def test_dispatch_from_8_bits(T, k, E, d, dt):
    say(f"case: dispatch from 8 bits T {T} k {k} E {E} d {d} {dt}")
    ids = choices(T, T, k, E)
    s = TokenSort(ids, E)
    o = RMSNorm(1 + rand(2, d, std=0.2)).forward(rand(1, T, d, std=2.0), y=False, mx=True)
    q, scale = o.q, o.scale
    q.view(torch.uint8)[0, 0] = 0x7f
    values = TR.mx_values(q, scale)
    rows = s.dispatch(q, scale=scale, dtype=DT[dt])
    want = values.float().to(DT[dt])[s.order.long() // k]
    want[int(s.offsets[-1]):] = 0
    assert torch.equal(torch.nan_to_num(rows, 7.0), torch.nan_to_num(want, 7.0))
    big = torch.zeros(T, d + 3, dtype=torch.uint8, device="cuda")  # rows at odd bytes
    big[:, 2:2 + d] = q.view(torch.uint8)
    again = s.dispatch(big.view(torch.float8_e4m3fn)[:, 2:2 + d], scale=scale, dtype=DT[dt])
    assert torch.equal(torch.nan_to_num(again, 7.0), torch.nan_to_num(want, 7.0))


@pytest.mark.parametrize("dt", DT)
def test_strides(dt):
    T, k, E, d, pad = 37, 3, 6, 101, 5
    dtype = DT[dt]
    ids = choices(1, T, k, E)
    s = TokenSort(ids, E)
    x, y, dout, gates = rand(1, T, d, dtype=dtype), rand(2, T * k, d, dtype=dtype), rand(3, T, d), rand(4, T, k)
    rows, buf = strided(torch.zeros(T * k, d, dtype=dtype, device="cuda"), pad, 3)
    assert torch.equal(s.dispatch(strided(x, 1, 1)[0], out=rows), s.dispatch(x))
    assert torch.isnan(buf[:3]).all() and torch.isnan(buf[3:].view(T * k, d + pad)[:, d:]).all()
    out, buf = strided(torch.zeros(T, d, device="cuda"), pad, 1)
    ys = strided(y, 3, 1)[0]
    assert torch.equal(s.combine(ys, gates, residual=strided(dout, 2, 3)[0], out=out), s.combine(y, gates, residual=dout))
    assert torch.isnan(buf[1:].view(T, d + pad)[:, d:]).all()
    for p, q in zip(s.combine_backward(ys, gates, strided(dout, 7, 1)[0]), s.combine_backward(y, gates, dout)):
        assert torch.equal(p, q)


def test_infinities_stay_in_their_rows():
    T, k, E, d = 20, 2, 4, 64
    ids = choices(5, T, k, E, none=0)
    s = TokenSort(ids, E)
    y = rand(1, T * k, d)
    clean = s.combine(y, rand(2, T, k))
    y[int(s.place[3, 1])] = float("inf")
    out = s.combine(y, rand(2, T, k))
    keep = torch.arange(T, device="cuda") != 3
    assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[3]).any()


def test_long_offsets():
    """Rows past 2^31 elements."""
    T, k, E, d = 70000, 8, 16, 4096
    ids = choices(9, T, k, E, none=0.01)
    s = TokenSort(ids, E)
    live = int(s.offsets[-1])
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    rows = s.dispatch(x)
    assert rows.numel() > 1 << 31
    at = torch.cat([torch.arange(0, 100), torch.arange(live - 200, live)]).cuda()
    assert torch.equal(rows[at], x[s.order[at].long() // k]) and not rows[live:].any()
    gates = torch.rand(T, k, device="cuda")
    out = s.combine(rows, gates)
    tail = slice(T - 50, T)
    w = torch.where(s.place < live, gates, 0.0)[tail].double()
    ref = (w[:, :, None] * x[tail].double()[:, None]).sum(1)
    size = (w[:, :, None] * x[tail].double()[:, None]).abs().sum(1)
    R.check("out", out[tail], R.rounded(ref, size * (k + 2) * TR.E23, torch.bfloat16))
    drows, dgates = s.combine_backward(rows, gates, x)
    sq = (x[tail].double() ** 2).sum(1, keepdim=True)
    ref = torch.where((s.place < live)[tail], sq, 0.0)
    R.check("dgates", dgates[tail], (ref, ref * 12 * TR.E23 + 1e-37))
    last = s.place[T - 1].long()
    want = torch.where(s.place[T - 1] < live, gates[T - 1], 0.0)[:, None] * x[T - 1].float()
    assert torch.equal(drows[last], want.to(torch.bfloat16))


def test_graph():
    T, k, E, d = 200, 4, 12, 520
    ids, x, gates, y = choices(1, T, k, E), rand(1, T, d), rand(2, T, k), rand(3, T * k, d)

    def step():
        s = TokenSort(ids, E)
        rows = s.dispatch(x)
        return [s.order, rows, s.combine(y, gates, residual=x), *s.combine_backward(y, gates, x), s.dispatch_backward(y)]

    for tokens in (T, 40):  # and the sort of several blocks
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                kept = step()
        torch.cuda.synchronize()
        for seed in range(4):
            ids.copy_(choices(20 + seed, T, k, E))
            x.copy_(rand(20 + seed, T, d))
            want = step()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(kept, want):
                assert torch.equal(p, q)
        T = 3000
        ids, x, gates, y = choices(1, T, k, E), rand(1, T, d), rand(2, T, k), rand(3, T * k, d)


def test_refusals():
    """What the Python side turns down before any call."""
    ids = choices(1, 6, 2, 4)
    s = TokenSort(ids, 4)
    x, rows, w = rand(1, 6, 16), rand(2, 12, 16), rand(3, 6, 2)
    bad = [lambda: TokenSort(ids.float(), 4), lambda: TokenSort(ids[:, :1].expand(6, 2), 4), lambda: TokenSort(ids[None], 4),
           lambda: s.dispatch(x[:5]), lambda: s.dispatch(x.double()), lambda: s.dispatch(x, dtype=torch.bfloat16),
           lambda: s.dispatch(x, scale=w), lambda: s.dispatch(x.cpu()), lambda: s.dispatch(x, out=rows[:11]),
           lambda: s.combine(rows[:11]), lambda: s.combine(rows, w.t().contiguous()), lambda: s.combine(rows, w.bfloat16()),
           lambda: s.combine(rows, w.view(-1)), lambda: s.combine(rows, torch.cat([w, w], 1)[:, :2]),
           lambda: s.combine(rows, out_dtype=torch.bfloat16), lambda: s.combine(rows, residual=x[:, :8]),
           lambda: s.combine_backward(rows, w, x.bfloat16()), lambda: s.combine_backward(rows, w, x[:5]),
           lambda: RMSNorm(x), lambda: RMSNorm(x[0], eps=-1.0), lambda: RMSNorm(x[0], sum_dtype=torch.bfloat16),
           lambda: RMSNorm(x[0]).forward(x, y=False), lambda: RMSNorm(x[0]).forward(x, sum_out=x),
           lambda: RMSNorm(x[0]).backward(x, None, x), lambda: RMSNorm(x[0]).backward(x, x[:, 0].contiguous(), x, ds=x, need_dx=False)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    for call in (lambda: TokenSort(ids, 0), lambda: TokenSort(ids, 1025), lambda: s.combine(rows, out=rows[:6])):
        with pytest.raises(ecf.EcfError):
            call()
