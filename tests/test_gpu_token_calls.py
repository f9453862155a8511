"""GPU tests of how the token operators' entry points are called: refusals, strides of ids, streams, graphs, a norm without a
weight."""
import pytest
import torch

import expert_cache_ffn_amd as ecf
from expert_cache_ffn_amd.layer import LowRankAdapters, RMSNorm, TokenSort
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


def whole_step(T, k=3, E=9, d=264, r=12, n=4):
    """A step of all token operators with workspaces (more than 8192 choices are sorted in two launches), from shared objects:
    (inputs of a seed, the step)."""
    norm = RMSNorm(1 + rand(1, d, std=0.1))
    adapters = LowRankAdapters(rand(2, n, r, d, std=d ** -.5), rand(3, n, d, r, std=r ** -.5), 0.5 + rand(4, n).abs())

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return dict(x=rand(seed, T, d), res=rand(seed + 1, T, d), dy=rand(seed + 2, T, d), gates=rand(seed + 3, T, k),
                    ids=torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).cuda(),
                    by=torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda())

    def step(q):
        o = norm.forward(q["x"], residual=q["res"], save=True)
        y, h = adapters.forward(o.y, q["by"], residual=o.y, save=True)
        s = TokenSort(q["ids"], E)
        rows = s.dispatch(y)
        out = s.combine(rows, q["gates"], residual=o.sum)
        drows, dgates = s.combine_backward(rows, q["gates"], q["dy"])
        dy = s.dispatch_backward(drows)
        dx, ddown, dup = adapters.backward(o.y, q["by"], h, dy, residual=dy)
        return [out, s.order, s.offsets, dgates, ddown, dup, *norm.backward(o.sum, o.rstd, dx, dsum=q["dy"])]

    return inputs, step


@pytest.mark.parametrize("T", [40, 200, 3000])
def test_two_streams_at_once(T):
    """Calls of the same objects on two streams share nothing."""
    inputs, step = whole_step(T)
    sets = [inputs(10), inputs(20)]
    want = [step(q) for q in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(step(sets[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            for p, q in zip(outs, want[i]):
                assert torch.equal(p, q)


@pytest.mark.parametrize("T", [40, 200, 3000])
def test_two_graphs(T):
    """Two captured graphs of the same objects, replayed one after the other and at once, with eager calls between."""
    inputs, step = whole_step(T)
    sets, graphs, kept = [inputs(10), inputs(20)], [], []
    for q in sets:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(q)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                kept.append(step(q))
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in range(4):
        for i, q in enumerate(sets):
            for name, v in inputs(100 * seed + 50 * i).items():
                q[name].copy_(v)
        want = [step(q) for q in sets]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            if seed % 2:
                graph.replay()
            else:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for outs, ref in zip(kept, want):
            for p, q in zip(outs, ref):
                assert torch.equal(p, q)


@pytest.mark.parametrize("T,d", [(5, 7), (70, 264), (9, 9000), (3, 20000)])
def test_a_norm_without_a_weight(T, d):
    """The C call without a weight, whose y and gradients are those of ones."""
    x, dy = rand(1, T, d), rand(2, T, d)
    norm = RMSNorm(torch.ones(d, device="cuda"))
    want = norm.forward(x, save=True)
    dx, _, dw = norm.backward(x, want.rstd, dy)
    a = ecf.NormArgs()
    a.hidden, a.eps, a.stream = d, norm._a.eps, torch.cuda.current_stream().cuda_stream or None
    y, rstd, dx2, dw2 = torch.empty_like(x), torch.empty_like(want.rstd), torch.empty_like(x), torch.empty_like(dw)
    a.d_x, a.d_y, a.d_rstd = x.data_ptr(), y.data_ptr(), rstd.data_ptr()
    ecf.ecf_norm_forward(a, T)
    ws = torch.empty(ecf.ecf_norm_workspace_bytes(d, T, True), dtype=torch.uint8, device="cuda")
    a.d_sum, a.d_dy, a.d_dx, a.d_dweight, a.d_ws, a.ws_bytes = (x.data_ptr(), dy.data_ptr(), dx2.data_ptr(), dw2.data_ptr(), ws.data_ptr(),
                                                                ws.numel())
    ecf.ecf_norm_backward(a, T)
    for p, q in ((y, want.y), (rstd, want.rstd), (dx2, dx), (dw2, dw)):
        assert torch.equal(p, q)
