"""CPU tests of the dense feed-forward operators' refusals and workspace sizes:
every bad call is turned down before any device work."""
import ctypes

import pytest
import torch

import expert_cache_ffn_amd as ecf
from expert_cache_ffn_amd import layer as ly

A = 1 << 20  # an address nothing dereferences: the calls below never reach a kernel


def gated(**kw):
    a = ecf.GatedArgs()
    a.hidden, a.inter, a.dtype, a.act, a.wgrad_dtype = 64, 32, ecf.ECF_BF16, ecf.ECF_ACT_SILU, ecf.ECF_BF16
    for f in ("d_x", "d_w_gate", "d_w_up", "d_h", "d_a", "d_b", "d_dh", "d_dx", "d_dw_gate", "d_dw_up"):
        setattr(a, f, A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def linear(**kw):
    a = ecf.LinearArgs()
    a.in_features, a.out_features, a.dtype, a.out_dtype, a.wgrad_dtype = 64, 32, ecf.ECF_BF16, ecf.ECF_F32, ecf.ECF_F32
    a.act = ecf.ECF_ACT_GELU
    for f in ("d_x", "d_w", "d_out", "d_z", "d_dout", "d_dx", "d_dw"):
        setattr(a, f, A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(fn, args, T=4, code=ecf.ECF_EINVAL):
    with pytest.raises(ecf.EcfError) as e:
        fn(args, T)
    assert e.value.code == code, str(e.value)


COMMON = [dict(dtype=ecf.ECF_MXFP4), dict(dtype=7), dict(act=5), dict(act=-1), dict(d_x=A + 1), dict(d_x=0), dict(ld_x=63)]


@pytest.mark.parametrize("bad", COMMON + [dict(hidden=0), dict(inter=-1), dict(hidden=(1 << 22) + 1), dict(d_w_gate=0),
                                          dict(d_w_up=A + 1), dict(d_h=0, d_a=0, d_b=0), dict(d_a=0), dict(d_b=0),
                                          dict(ld_w=10), dict(ld_h=31), dict(ld_ab=-5), dict(d_b_gate=A + 1)])
def test_gated_forward_refusals(bad):
    refused(ecf.ecf_gated_forward, gated(**bad))


@pytest.mark.parametrize("bad", COMMON + [dict(inter=0), dict(d_a=0), dict(d_b=A + 1), dict(d_dh=0), dict(ld_dh=1),
                                          dict(wgrad_dtype=ecf.ECF_F16), dict(d_dw_up=0), dict(ld_dw=63),
                                          dict(d_dx=A + 1), dict(d_db_up=A + 1), dict(d_w_gate=0)])
def test_gated_backward_refusals(bad):
    refused(ecf.ecf_gated_backward, gated(d_ws=A, ws_bytes=1 << 30, **bad))


@pytest.mark.parametrize("bad", COMMON + [dict(in_features=0), dict(out_dtype=ecf.ECF_F16), dict(d_w=0), dict(d_out=0),
                                          dict(d_out=A + 2), dict(d_z=A + 1), dict(d_residual=A + 2), dict(ld_out=31),
                                          dict(ld_residual=31, d_residual=A), dict(d_bias=A + 1)])
def test_linear_forward_refusals(bad):
    refused(ecf.ecf_linear_forward, linear(**bad))


@pytest.mark.parametrize("bad", COMMON + [dict(out_features=0), dict(d_z=0), dict(d_dout=A + 2), dict(d_dout=0),
                                          dict(d_dw=A + 2), dict(wgrad_dtype=ecf.ECF_MXFP4), dict(d_dbias=A + 2),
                                          dict(ld_dout=31), dict(ld_dx=63)])
def test_linear_backward_refusals(bad):
    refused(ecf.ecf_linear_backward, linear(d_ws=A, ws_bytes=1 << 30, **bad))


def test_token_counts_and_null():
    for fn, args in ((ecf.ecf_gated_forward, gated), (ecf.ecf_gated_backward, gated), (ecf.ecf_linear_forward, linear),
                     (ecf.ecf_linear_backward, linear)):
        refused(fn, args(), T=-1)
        refused(fn, args(), T=(1 << 22) + 1)
    for name in ("ecf_gated_forward", "ecf_gated_backward", "ecf_linear_forward", "ecf_linear_backward"):
        assert getattr(ecf.lib(), name)(None, 4) == ecf.ECF_EINVAL
    # no tokens: a forward call has nothing to do and looks at no pointer
    ecf.ecf_gated_forward(gated(d_x=0, d_h=0, d_a=0, d_b=0), 0)
    ecf.ecf_linear_forward(linear(d_x=0, d_out=0), 0)


def test_workspace():
    for fn, args, size in ((ecf.ecf_gated_backward, gated, ecf.ecf_gated_workspace_bytes),
                           (ecf.ecf_linear_backward, linear, ecf.ecf_linear_workspace_bytes)):
        need = size(64, 32, ecf.ECF_BF16, 100, True)
        assert need > 0
        refused(fn, args(), T=100, code=ecf.ECF_ENOSPC)
        refused(fn, args(d_ws=A, ws_bytes=need - 1), T=100, code=ecf.ECF_ENOSPC)
        refused(fn, args(d_ws=A + 128, ws_bytes=need), T=100)
        # monotone in the tokens, for both directions and every type
        for back in (False, True):
            for dt in (ecf.ECF_F32, ecf.ECF_BF16, ecf.ECF_F16):
                last = 0
                for T in (0, 1, 2, 8, 16, 17, 33, 64, 100, 128, 129, 500, 1000, 4096, 8192, 100000):
                    n = size(4096, 1024, dt, T, back)
                    assert n >= last, (T, n, last)
                    last = n
        for bad in ((0, 32, ecf.ECF_BF16, 4), (64, 1 << 23, ecf.ECF_BF16, 4), (64, 32, ecf.ECF_MXFP4, 4),
                    (64, 32, ecf.ECF_BF16, -1)):
            with pytest.raises(ecf.EcfError):
                size(*bad, True)


def test_long_strides_are_refused():
    ld = (1 << 31) // 256 // 2
    refused(ecf.ecf_gated_forward, gated(ld_x=ld), code=ecf.ECF_EUNSUPPORTED)
    refused(ecf.ecf_linear_forward, linear(ld_out=ld), code=ecf.ECF_EUNSUPPORTED)
    refused(ecf.ecf_linear_backward, linear(ld_z=ld, d_ws=A, ws_bytes=1 << 30), code=ecf.ECF_EUNSUPPORTED)


def test_fp16_stays_out_of_the_moe_layer():
    for w, a in ((ecf.ECF_F16, ecf.ECF_BF16), (ecf.ECF_BF16, ecf.ECF_F16), (ecf.ECF_F16, ecf.ECF_F16)):
        with pytest.raises(ecf.EcfError):
            ecf.ecf_expert_bytes(ecf.make_shape(256, 64, 4, 2, w, a))


def test_python_argument_checks():
    w = torch.zeros(8, 16)
    for make in (lambda: ly.Linear(w), lambda: ly.GatedProjection(w, w)):  # not on the GPU
        with pytest.raises(ValueError):
            make()
    dev = w.device
    with pytest.raises(ValueError):
        ly._matrix("x", w, 8, 17, torch.float32, dev)
    with pytest.raises(ValueError):
        ly._matrix("x", w, 8, 16, torch.bfloat16, dev)
    with pytest.raises(ValueError):
        ly._matrix("x", w.t(), 16, 8, torch.float32, dev)
    with pytest.raises(ValueError):  # a broadcast tensor's rows are the same memory
        ly._matrix("x", w[:1].expand(8, 16), 8, 16, torch.float32, dev)
    assert ly._matrix("x", w[:, 3:9], 8, 6, torch.float32, dev) == (w.data_ptr() + 12, 16)
    assert ly._matrix("x", w[2:3], 1, 16, torch.float32, dev)[1] == 16
    with pytest.raises(ValueError):
        ly._vector("b", torch.zeros(16)[::2], 8, torch.float32, dev)
    assert ctypes.sizeof(ecf.GatedArgs) == 216 and ctypes.sizeof(ecf.LinearArgs) == 200


DISTINCT = {f: A + 4096 * i for i, f in enumerate(
    ("d_x", "d_w", "d_w_gate", "d_w_up", "d_b_gate", "d_b_up", "d_bias", "d_h", "d_a", "d_b", "d_z", "d_dh", "d_dout", "d_out",
     "d_residual", "d_dx", "d_dw", "d_dw_gate", "d_dw_up", "d_db_gate", "d_db_up", "d_dbias", "d_ws"))}


@pytest.mark.parametrize("fn,make,out,others", [
    (ecf.ecf_gated_forward, gated, "d_h", ("d_x", "d_w_gate", "d_w_up", "d_a", "d_b", "d_b_up")),
    (ecf.ecf_gated_forward, gated, "d_b", ("d_x", "d_a", "d_h", "d_w_up")),
    (ecf.ecf_gated_backward, gated, "d_dx", ("d_x", "d_a", "d_b", "d_dh", "d_w_gate", "d_dw_up")),
    (ecf.ecf_gated_backward, gated, "d_dw_gate", ("d_x", "d_w_gate", "d_dw_up", "d_db_up", "d_ws")),
    (ecf.ecf_linear_forward, linear, "d_out", ("d_x", "d_w", "d_bias", "d_z")),
    (ecf.ecf_linear_forward, linear, "d_z", ("d_x", "d_residual")),
    (ecf.ecf_linear_backward, linear, "d_dx", ("d_x", "d_z", "d_dout", "d_w", "d_dw", "d_dbias")),
    (ecf.ecf_linear_backward, linear, "d_dw", ("d_w", "d_x", "d_dbias"))])
def test_outputs_on_other_operands_are_refused(fn, make, out, others):
    for other in others:
        args = make(ws_bytes=1 << 30)
        for f in DISTINCT:
            if hasattr(args, f):
                setattr(args, f, DISTINCT[f])
        setattr(args, out, getattr(args, other))
        with pytest.raises(ecf.EcfError, match="same memory") as e:
            fn(args, 4)
        assert e.value.code == ecf.ECF_EINVAL


def test_residual_in_place_needs_its_stride():
    args = linear(d_x=A, d_w=2 * A, d_out=3 * A, d_residual=3 * A, d_z=0, ld_out=40, ld_residual=48)
    refused(ecf.ecf_linear_forward, args)


def test_few_tokens_need_no_workspace():
    """Up to 16 tokens and 2^17 elements of x (a captured decode step needs no buffer for it)."""
    for dt in (ecf.ECF_F32, ecf.ECF_BF16, ecf.ECF_F16):
        for T, K in ((1, 1), (1, 4096), (16, 4096), (1, 100000)):
            if K == 1 and dt != ecf.ECF_F32:
                continue  # 16-bit rows of odd length
            assert ecf.ecf_gated_workspace_bytes(K, 1024, dt, T) == 0
            assert ecf.ecf_linear_workspace_bytes(K, 1024, dt, T) == 0
        assert ecf.ecf_linear_workspace_bytes(8192, 1024, dt, 16) > 0
        assert ecf.ecf_linear_workspace_bytes(4096, 1024, dt, 17) > 0


def test_lost_gradients_are_said(recwarn):
    with torch.no_grad():
        ly._warn_untracked("Linear")
    assert not recwarn.list
    with pytest.warns(UserWarning, match="Linear.forward is outside autograd"):
        ly._warn_untracked("Linear")
