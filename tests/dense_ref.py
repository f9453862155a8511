"""64-bit reference of the dense feed-forward operators, with an elementwise
bound on how far a right kernel may be from it.

The bounds count, for each output:
  * its own rounding, half a step of its type (eps / 2 relative; in fp16 half a
    subnormal step where that is more);
  * fp32 sums of n products: any order of adding n terms, each addition off by at
    most one fp32 step (2^-23, so that truncating adders are covered too), is
    within n 2^-23 of the sum of the absolute products;
  * the activation in fp32: 32 steps for the functions themselves plus what the
    rounding of their argument moves them by (relative change of the result per
    relative change of the argument: |u2| <= 2 (|v| + 0.1 |v|^3) for the
    sigmoid forms, v^2 for erfc), so (32 + 4 v^2 + 8 |v| + |v|^3) 2^-23;
  * in the backward passes, da, db and dz rounded once to the operands' type.
"""
import math

import torch

EPS23 = 2.0 ** -23
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -126}


def act_both(v, act):
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return v.clamp_min(0), (v > 0).double()
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * torch.sigmoid(-v)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
    return v * p, p + v * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * v * v)


def act_rel(v):
    return (32 + 4 * v * v + 8 * v.abs() + v.abs() ** 3) * EPS23


def half_step(ref, dtype):
    return ref.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def product(a, b, da=None):
    """a @ b^T with its bound: a [M, K] (known to within da), b [N, K]."""
    z = a @ b.t()
    err = (a.abs() @ b.abs().t()) * ((a.shape[1] + 2) * EPS23)
    if da is not None:
        err = err + da @ b.abs().t() * (1 + a.shape[1] * EPS23)
    return z, err


def with_bias(z, err, bias):
    if bias is None:
        return z, err
    return z + bias, err + (z + bias).abs() * EPS23


def through_act(z, err, act):
    """(value, bound); every activation's slope is at most 1.2."""
    v, _ = act_both(z, act)
    if act == "none":
        return v, err
    return v, 1.2 * err + act_rel(z) * v.abs() + 1e-37


def gated_forward(x, wg, wu, bg, bu, act, dtype):
    """{name: (reference, bound)} of h, a and b."""
    a, ea = with_bias(*product(x, wg), bg)
    b, eb = with_bias(*product(x, wu), bu)
    v, ev = through_act(a, ea, act)
    h = v * b
    eh = ev * b.abs() + v.abs() * eb + ev * eb + h.abs() * EPS23
    r = {"h": (h, eh), "a": (a, ea), "b": (b, eb)}
    return {k: (ref, e + half_step(ref, dtype) * (1 + 1e-3)) for k, (ref, e) in r.items()}


def grads(dout, z, act, dtype, b=None):
    """dz (linear) or da, db (gated) before and after rounding: [(value, bound of the
    unrounded value, bound of the rounded one)]."""
    v, s = act_both(z, act)
    rel = act_rel(z) if act not in ("none", "relu") else torch.zeros_like(z)
    # the slope is a sum of two terms of either sign, each within rel of its size
    size = s.abs() if act in ("none", "relu") else 1 + z.abs()
    out = []
    d = dout * s * (1 if b is None else b)
    e = (dout * (1 if b is None else b)).abs() * size * (rel + 3 * EPS23) if act != "none" or b is not None \
        else torch.zeros_like(d)
    out.append((d, e, e + half_step(d, dtype) * (1 + 1e-3)))
    if b is not None:
        d = dout * v
        e = d.abs() * (rel + 2 * EPS23) + dout.abs() * 1e-37
        out.append((d, e, e + half_step(d, dtype) * (1 + 1e-3)))
    return out


def colsum(d, e, gd):
    s = d.sum(0)
    err = e.sum(0) + (d.shape[0] + 2) * EPS23 * d.abs().sum(0)
    return s, err + half_step(s, gd) * (1 + 1e-3)


def rounded(ref, err, dtype):
    return ref, err + half_step(ref, dtype) * (1 + 1e-3)


def gated_backward(x, wg, wu, a, b, dh, act, dtype, gd):
    (da, ea, ra), (db, eb, rb) = grads(dh, a, act, dtype, b)
    dx, ex = product(torch.cat([da, db], 1), torch.cat([wg, wu], 0).t().contiguous(), torch.cat([ra, rb], 1))
    r = {"dx": rounded(dx, ex, dtype)}
    for n, d, q in (("dw_gate", da, ra), ("dw_up", db, rb)):
        r[n] = rounded(*product(d.t(), x.t(), q.t()), gd)
    r["db_gate"], r["db_up"] = colsum(da, ea, gd), colsum(db, eb, gd)
    return r


def linear_forward(x, w, bias, act, residual, dtype, out_dtype):
    z, ez = with_bias(*product(x, w), bias)
    y, ey = through_act(z, ez, act)
    if residual is not None:
        y = y + residual
        ey = ey + y.abs() * EPS23
    return {"y": rounded(y, ey, out_dtype), "z": rounded(z, ez, dtype)}


def linear_backward(x, w, z, dout, act, dtype, out_dtype, gd):
    (dz, e, r), = grads(dout, dout if z is None else z, act, dtype)
    if act == "none" and dtype == out_dtype:
        r = torch.zeros_like(dz)  # dy itself
    return {"dx": rounded(*product(dz, w.t().contiguous(), r), dtype),
            "dw": rounded(*product(dz.t(), x.t(), r.t()), gd),
            "dbias": colsum(dz, e, gd)}


def check(name, got, ref_bound):
    ref, bound = (v.to(got.device) for v in ref_bound)
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)}, want {tuple(ref.shape)}"
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got "
                             f"{float(got[i])!r}, want {float(ref[i])!r} +- {float(bound[i]):.3g}")
