"""CPU tests of the token operators' refusals and workspace sizes: every bad call is turned down
before any device work."""
import ctypes

import pytest
import torch

import expert_cache_ffn_amd as ecf
from expert_cache_ffn_amd import layer as ly

A = 1 << 20  # an address nothing dereferences: the calls below never reach a kernel


def fill(a, names, **kw):
    for i, f in enumerate(names):
        setattr(a, f, A + 4096 * i)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm_fwd(**kw):
    a = ecf.NormArgs()
    a.hidden, a.dtype, a.sum_dtype, a.weight_dtype, a.eps = 64, ecf.ECF_BF16, ecf.ECF_F32, ecf.ECF_BF16, 1e-6
    return fill(a, ("d_weight", "d_x", "d_residual", "d_sum", "d_y", "d_q", "d_q_scale", "d_rstd"), **kw)


def norm_bwd(**kw):
    a = ecf.NormArgs()
    a.hidden, a.dtype, a.sum_dtype, a.weight_dtype, a.wgrad_dtype = 64, ecf.ECF_BF16, ecf.ECF_F32, ecf.ECF_BF16, ecf.ECF_F32
    a.ws_bytes = 1 << 30
    return fill(a, ("d_weight", "d_sum", "d_rstd", "d_dy", "d_dsum", "d_dx", "d_ds", "d_dweight", "d_ws"), **kw)


def sort(**kw):
    a = ecf.SortArgs()
    a.n_experts, a.top_k, a.idx_bytes, a.ws_bytes = 8, 2, 4, 1 << 30
    return fill(a, ("d_idx", "d_counts", "d_offsets", "d_tiles", "d_order", "d_place", "d_ws"), **kw)


def move(**kw):
    a = ecf.TokenArgs()
    a.hidden, a.n_experts, a.top_k, a.dtype, a.token_dtype = 64, 8, 2, ecf.ECF_BF16, ecf.ECF_BF16
    return fill(a, ("d_offsets", "d_place", "d_weight", "d_x", "d_x_scale", "d_rows", "d_residual", "d_out", "d_dout",
                    "d_drows", "d_dweight"), **kw)


def refused(fn, args, T=4, code=ecf.ECF_EINVAL, match=None):
    with pytest.raises(ecf.EcfError, match=match) as e:
        fn(args, T)
    assert e.value.code == code, str(e.value)


NORM = [dict(hidden=0), dict(hidden=(1 << 22) + 1), dict(dtype=ecf.ECF_MXFP4), dict(dtype=ecf.ECF_MXFP8), dict(dtype=9),
        dict(sum_dtype=ecf.ECF_F16), dict(weight_dtype=ecf.ECF_F16), dict(eps=-1.0), dict(eps=float("nan")),
        dict(eps=float("inf")), dict(d_weight=A + 1)]


@pytest.mark.parametrize("bad", NORM + [dict(d_x=0), dict(d_x=A + 1), dict(ld_x=63), dict(d_residual=A + 2), dict(ld_residual=60),
                                        dict(d_residual=0), dict(ld_sum=63), dict(d_y=0, d_q=0, d_q_scale=0), dict(d_y=A + 1),
                                        dict(ld_y=1), dict(d_q=0), dict(d_q_scale=0), dict(ld_q=63), dict(ld_q_scale=1),
                                        dict(d_rstd=A + 2)])
def test_norm_forward_refusals(bad):
    refused(ecf.ecf_norm_forward, norm_fwd(**bad))


@pytest.mark.parametrize("bad", NORM + [dict(wgrad_dtype=ecf.ECF_F16), dict(d_sum=0), dict(d_sum=A + 2), dict(ld_sum=8), dict(d_rstd=0),
                                        dict(d_dy=0), dict(ld_dy=63), dict(d_dsum=A + 2), dict(ld_dsum=63), dict(d_dx=A + 1),
                                        dict(ld_dx=63), dict(d_ds=A + 2), dict(ld_ds=63), dict(d_dweight=A + 2)])
def test_norm_backward_refusals(bad):
    refused(ecf.ecf_norm_backward, norm_bwd(**bad))


SHAPE = [dict(n_experts=0), dict(n_experts=1025), dict(top_k=0), dict(top_k=33)]


@pytest.mark.parametrize("bad", SHAPE + [dict(idx_bytes=2), dict(d_idx=0), dict(d_idx=A + 2), dict(ld_idx=1), dict(d_counts=0),
                                         dict(d_offsets=A + 1), dict(d_tiles=0), dict(d_order=0), dict(d_place=A + 2)])
def test_sort_refusals(bad):
    refused(ecf.ecf_token_sort, sort(**bad))


MOVE = SHAPE + [dict(hidden=0), dict(dtype=ecf.ECF_MXFP8), dict(dtype=ecf.ECF_MXFP4), dict(token_dtype=ecf.ECF_F16), dict(d_offsets=0),
                dict(d_place=0), dict(d_weight=A + 2), dict(d_rows=A + 1), dict(ld_rows=63)]


@pytest.mark.parametrize("bad", MOVE + [dict(token_dtype=ecf.ECF_F32), dict(d_x=0), dict(ld_x=63), dict(d_rows=0),
                                        dict(token_dtype=ecf.ECF_MXFP8, d_x_scale=0),
                                        dict(token_dtype=ecf.ECF_MXFP8, ld_x_scale=1)])
def test_dispatch_refusals(bad):
    refused(ecf.ecf_token_dispatch, move(**bad))


@pytest.mark.parametrize("bad", MOVE + [dict(token_dtype=ecf.ECF_MXFP8), dict(d_rows=0), dict(d_out=0), dict(d_out=A + 1), dict(ld_out=2),
                                        dict(d_residual=A + 1), dict(ld_residual=63)])
def test_combine_refusals(bad):
    refused(ecf.ecf_token_combine, move(**bad))


@pytest.mark.parametrize("bad", MOVE + [dict(token_dtype=ecf.ECF_MXFP8), dict(d_rows=0), dict(d_dout=0), dict(ld_dout=1),
                                        dict(d_drows=A + 1), dict(ld_drows=63), dict(d_dweight=A + 2)])
def test_combine_backward_refusals(bad):
    refused(ecf.ecf_token_combine_backward, move(**bad))


CALLS = [(ecf.ecf_norm_forward, norm_fwd), (ecf.ecf_norm_backward, norm_bwd), (ecf.ecf_token_sort, sort), (ecf.ecf_token_dispatch, move),
         (ecf.ecf_token_combine, move), (ecf.ecf_token_combine_backward, move)]


@pytest.mark.parametrize("fn,make", CALLS)
def test_token_counts_and_null(fn, make):
    refused(fn, make(), T=-1)
    refused(fn, make(), T=(1 << 22) + 1)
    assert getattr(ecf.lib(), fn.__name__)(None, 4) == ecf.ECF_EINVAL


def test_too_many_choices():
    refused(ecf.ecf_token_sort, sort(top_k=32), T=(1 << 21) + 1)
    refused(ecf.ecf_token_combine, move(top_k=32), T=(1 << 21) + 1)


def test_no_tokens_look_at_no_pointer():
    ecf.ecf_norm_forward(norm_fwd(d_x=0, d_y=0), 0)
    for fn in (ecf.ecf_token_dispatch, ecf.ecf_token_combine, ecf.ecf_token_combine_backward):
        fn(move(d_x=0, d_rows=0, d_out=0, d_dout=0, d_place=0, d_offsets=0), 0)


def test_long_strides_are_refused():
    ld = 1 << 31
    refused(ecf.ecf_norm_forward, norm_fwd(ld_x=ld), code=ecf.ECF_EUNSUPPORTED)
    refused(ecf.ecf_token_combine, move(ld_rows=ld), code=ecf.ECF_EUNSUPPORTED)


@pytest.mark.parametrize("fn,make,out,others", [
    (ecf.ecf_norm_forward, norm_fwd, "d_sum", ("d_x", "d_weight", "d_y", "d_q")),
    (ecf.ecf_norm_forward, norm_fwd, "d_y", ("d_x", "d_residual", "d_sum", "d_weight", "d_q", "d_rstd")),
    (ecf.ecf_norm_forward, norm_fwd, "d_q_scale", ("d_x", "d_residual", "d_q")),
    (ecf.ecf_norm_backward, norm_bwd, "d_dx", ("d_sum", "d_rstd", "d_dy", "d_dsum", "d_ds", "d_dweight", "d_weight", "d_ws")),
    (ecf.ecf_norm_backward, norm_bwd, "d_ds", ("d_sum", "d_dy", "d_ws")),
    (ecf.ecf_token_sort, sort, "d_order", ("d_idx", "d_counts", "d_offsets", "d_tiles", "d_place")),
    (ecf.ecf_token_dispatch, move, "d_rows", ("d_x", "d_offsets", "d_place")),
    (ecf.ecf_token_combine, move, "d_out", ("d_rows", "d_weight", "d_offsets", "d_place")),
    (ecf.ecf_token_combine_backward, move, "d_drows", ("d_dout", "d_rows", "d_weight", "d_dweight", "d_place"))])
def test_outputs_on_other_operands_are_refused(fn, make, out, others):
    for other in others:
        a = make()
        setattr(a, out, getattr(a, other))
        refused(fn, a, match="same memory")


def test_in_place_needs_its_stride():
    refused(ecf.ecf_norm_forward, norm_fwd(d_sum=A, d_residual=A, d_x=9 * A, d_weight=0, ld_sum=72, ld_residual=80), match="stride")
    refused(ecf.ecf_norm_backward, norm_bwd(d_ds=A, d_dsum=A, d_weight=0, d_sum=9 * A, ld_ds=72, ld_dsum=80), match="stride")
    refused(ecf.ecf_token_combine, move(d_out=9 * A, d_residual=9 * A, ld_out=72, ld_residual=80), match="stride")


def test_workspace():
    need = ecf.ecf_norm_workspace_bytes(64, 100, True)
    assert need == 100 * 64 * 4 and ecf.ecf_norm_workspace_bytes(64, 100) == 0
    refused(ecf.ecf_norm_backward, norm_bwd(ws_bytes=need - 1), T=100, code=ecf.ECF_ENOSPC)
    refused(ecf.ecf_norm_backward, norm_bwd(d_ws=A + 128), T=100)
    need = ecf.ecf_token_sort_workspace_bytes(8, 2, 50000)
    assert need > 0 and ecf.ecf_token_sort_workspace_bytes(8, 2, 2048) == 0
    refused(ecf.ecf_token_sort, sort(ws_bytes=need - 1), T=50000, code=ecf.ECF_ENOSPC)
    for size, shape in ((ecf.ecf_norm_workspace_bytes, (4096,)), (ecf.ecf_token_sort_workspace_bytes, (256, 6))):
        last = 0
        for T in (0, 1, 16, 500, 700, 5000, 100000, 1 << 22):
            n = size(*shape, T, True) if len(shape) == 1 else size(*shape, T)
            assert n >= last
            last = n
    for size, bad in ((ecf.ecf_norm_workspace_bytes, (0, 4, True)), (ecf.ecf_token_sort_workspace_bytes, (0, 2, 4))):
        with pytest.raises(ecf.EcfError):
            size(*bad)


def test_python_argument_checks():
    w = torch.ones(8)
    for make in (lambda: ly.RMSNorm(w), lambda: ly.TokenSort(torch.zeros(4, 2, dtype=torch.int32), 3)):  # not on the GPU
        with pytest.raises(ValueError):
            make()
    assert (ctypes.sizeof(ecf.NormArgs), ctypes.sizeof(ecf.SortArgs), ctypes.sizeof(ecf.TokenArgs)) == (240, 96, 176)


def adapter(**kw):
    a = ecf.AdapterArgs()
    a.in_features, a.out_features, a.rank, a.n_adapters, a.idx_bytes = 64, 32, 8, 4, 4
    a.dtype, a.out_dtype, a.wgrad_dtype, a.ws_bytes = ecf.ECF_BF16, ecf.ECF_F32, ecf.ECF_BF16, 1 << 30
    return fill(a, ("d_a", "d_b", "d_scale", "d_idx", "d_order", "d_offsets", "d_tiles", "d_x", "d_h", "d_residual", "d_out", "d_dout",
                    "d_dx", "d_da", "d_db", "d_ws"), **kw)


ADAPTER = [dict(in_features=0), dict(out_features=(1 << 22) + 1), dict(rank=0), dict(rank=257), dict(n_adapters=0), dict(n_adapters=1025),
           dict(dtype=ecf.ECF_MXFP8), dict(out_dtype=ecf.ECF_F16), dict(idx_bytes=2), dict(d_order=0), dict(d_offsets=0), dict(d_tiles=0),
           dict(d_order=A + 2), dict(d_scale=A + 2), dict(d_h=A + 1), dict(d_idx=0), dict(d_idx=A + 2), dict(d_b=0), dict(d_b=A + 1),
           dict(d_a=0), dict(d_x=0), dict(ld_x=63)]


@pytest.mark.parametrize("bad", ADAPTER + [dict(d_out=0), dict(d_out=A + 2), dict(ld_out=31), dict(d_residual=A + 2), dict(ld_residual=31)])
def test_adapter_forward_refusals(bad):
    refused(ecf.ecf_adapter_forward, adapter(**bad))


@pytest.mark.parametrize("bad", ADAPTER + [dict(d_dout=0), dict(d_dout=A + 2), dict(ld_dout=31), dict(d_h=0), dict(d_dx=A + 1), dict(ld_dx=63),
                                           dict(d_residual=A + 1), dict(ld_residual=63), dict(d_da=A + 1), dict(d_db=A + 1),
                                           dict(wgrad_dtype=ecf.ECF_F16)])
def test_adapter_backward_refusals(bad):
    refused(ecf.ecf_adapter_backward, adapter(**bad))


@pytest.mark.parametrize("fn,out,others", [
    (ecf.ecf_adapter_forward, "d_out", ("d_x", "d_a", "d_b", "d_scale", "d_idx", "d_order", "d_offsets", "d_tiles", "d_h")),
    (ecf.ecf_adapter_forward, "d_h", ("d_x", "d_residual")),
    (ecf.ecf_adapter_backward, "d_dx", ("d_x", "d_a", "d_dout", "d_h", "d_da", "d_db", "d_ws")),
    (ecf.ecf_adapter_backward, "d_db", ("d_b", "d_dout", "d_residual", "d_da", "d_order"))])
def test_adapter_outputs_on_other_operands_are_refused(fn, out, others):
    for other in others:
        a = adapter()
        setattr(a, out, getattr(a, other))
        refused(fn, a, match="same memory")


def test_adapter_counts_strides_and_workspace():
    for fn in (ecf.ecf_adapter_forward, ecf.ecf_adapter_backward):
        refused(fn, adapter(), T=-1)
        refused(fn, adapter(), T=(1 << 22) + 1)
        refused(fn, adapter(ws_bytes=100), T=100, code=ecf.ECF_ENOSPC)
        refused(fn, adapter(d_ws=adapter().d_x), T=100, match="256-byte|same memory")
        refused(fn, adapter(d_ws=A + 128), T=100)
        assert getattr(ecf.lib(), fn.__name__)(None, 4) == ecf.ECF_EINVAL
    refused(ecf.ecf_adapter_forward, adapter(ld_out=1 << 31), code=ecf.ECF_EUNSUPPORTED)
    refused(ecf.ecf_adapter_forward, adapter(d_out=9 * A, d_residual=9 * A, ld_out=40, ld_residual=48), match="stride")
    refused(ecf.ecf_adapter_backward, adapter(d_dx=9 * A, d_residual=9 * A, ld_dx=72, ld_residual=80), match="stride")
    ecf.ecf_adapter_forward(adapter(d_x=0, d_out=0, d_idx=0), 0)
    # a decode batch of small adapters needs no buffer
    assert ecf.ecf_adapter_workspace_bytes(4096, 4096, 16, 64, 16) == 0 < ecf.ecf_adapter_workspace_bytes(4096, 4096, 64, 64, 16)
    for bad in ((0, 32, 8, 4, 10), (64, 32, 300, 4, 10), (64, 32, 8, 4, -1)):
        with pytest.raises(ecf.EcfError):
            ecf.ecf_adapter_workspace_bytes(*bad)
    for back in (False, True):  # what serves so many tokens serves fewer
        for shape in ((4096, 4096, 16, 64), (64, 100, 3, 1), (300, 8192, 256, 1024)):
            last = 0
            for T in sorted({0, 1, 63, 64, 65, 100, 100000, 1 << 20} | {64 * i + d for i in range(1, 600, 7) for d in (-1, 0, 1)}):
                need = ecf.ecf_adapter_workspace_bytes(*shape, T, back)
                assert need >= last, (shape, T)
                last = need
    assert ctypes.sizeof(ecf.AdapterArgs) == 224
    with pytest.raises(ValueError):
        ly.LowRankAdapters(torch.zeros(2, 4, 8), torch.zeros(2, 8, 4))  # not on the GPU


def test_8_bits_stay_out_of_the_other_operators():
    for w, a in ((ecf.ECF_MXFP8, ecf.ECF_BF16), (ecf.ECF_BF16, ecf.ECF_MXFP8), (ecf.ECF_MXFP8, ecf.ECF_MXFP8)):
        with pytest.raises(ecf.EcfError):
            ecf.ecf_expert_bytes(ecf.make_shape(256, 64, 4, 2, w, a))
    with pytest.raises(ecf.EcfError):
        ecf.ecf_linear_workspace_bytes(64, 32, ecf.ECF_MXFP8, 4)
