"""64-bit references of the token operators, with elementwise bounds on how far a right
kernel may be from them.  E23 is one fp32 step (twice the rounding error, so that any way
of adding is covered); every output adds half a step of its own type."""
import torch

from dense_ref import EPS23 as E23
from dense_ref import half_step, rounded

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rand(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def strided(t, pad, shift):
    """The same values in rows `pad` elements further apart, starting `shift` elements in; the gaps
    hold NaN.  Returns (view, whole buffer)."""
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((rows * ld + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v, buf


def norm_sum(x, residual):
    """One fp32 addition, rounded to the residual's type: exact."""
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def norm_forward(total, weight, eps, dtype):
    """{y, rstd}: rstd is rounded to fp32 once, y is two fp32 products of it."""
    s = total.double()
    rstd = 1 / torch.sqrt((s * s).mean(1) + eps)
    y = s * rstd[:, None] * (1 if weight is None else weight.double())
    return {"y": rounded(y, 2 * E23 * y.abs(), dtype), "rstd": (rstd, E23 * rstd), "exact": (y, 2 * E23 * y.abs())}


def norm_backward(total, rstd, weight, dy, dsum, dtype, sum_dtype, gd):
    s, r, g = total.double(), rstd.double()[:, None], dy.double()
    h = s * r
    dw = (g * h).sum(0)
    edw = (g * h).abs().sum(0) * (len(s) + 4) * E23  # a sum over the rows in any order
    g = g * (1 if weight is None else weight.double())
    mean, size = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    past = 0 if dsum is None else dsum.double()
    v = past + r * (g - h * mean)
    # g and h are a product each, the mean's terms are added in fp32 eight at a time
    ev = E23 * (r * (3 * g.abs() + h.abs() * (12 * size + 3 * mean.abs())) + v.abs())
    return {"dx": rounded(v, ev, dtype), "ds": rounded(v, ev, sum_dtype), "dw": rounded(dw, edw, gd)}


def mx_bytes(y):
    """The scales' bytes of y [t, d] by the definition, in 64 bits."""
    t, d = y.shape
    n = (d + 31) // 32
    a = torch.nn.functional.pad(y.double().abs(), (0, n * 32 - d)).view(t, n, 32)
    top = torch.where(torch.isfinite(a), a, 0.0).amax(2)
    m, e = torch.frexp(top)  # m 2^e, m in [0.5, 1): 448 is 0.875 2^9
    return torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8) + 127, 0).clamp(0, 254)


def mx_values(q, scale):
    return q.double() * torch.exp2(scale.view(torch.uint8).double() - 127).repeat_interleave(32, dim=1)[:, : q.shape[1]]


def check_mx(q, scale, exact):
    """q and scale against y known to within a bound: a scale that is the least for some value within it, elements within
    half a step (2^-4 relative, 2^-10 of the scale below e4m3's normal numbers)."""
    y, e = exact
    b = scale.view(torch.uint8).long()
    lo, hi = mx_bytes((y.abs() - e).clamp_min(0)), mx_bytes(y.abs() + e)
    assert ((b >= lo) & (b <= hi)).all(), "a scale is not the least that holds its group"
    s = torch.exp2(b.double() - 127).repeat_interleave(32, dim=1)[:, : y.shape[1]]
    off = (mx_values(q, scale) - y).abs()
    assert (off <= torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) + e).all(), "an element is over half a step off"


def sort(ids, n):
    """(counts, offsets, order, place) on the CPU."""
    flat = ids.reshape(-1).cpu().long()
    keys = torch.where((flat >= 0) & (flat < n), flat, n)
    order = torch.argsort(keys, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order))
    counts = torch.bincount(keys, minlength=n + 1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts[:n].cumsum(0)])
    tiles = torch.cat([torch.zeros(1, dtype=torch.long), ((counts + 63) // 64).cumsum(0)])
    return {"counts": counts[:n], "offsets": offsets, "tiles": tiles, "order": order, "place": place.view(ids.shape[0], -1)}


def combine(rows, place, live, weights, residual, out_dtype):
    """live: rows of any expert."""
    y = torch.where(torch.arange(len(rows), device=rows.device)[:, None] < live, rows.double(), 0.0)[place.long()]
    w = torch.ones(place.shape, dtype=torch.float64, device=rows.device) if weights is None else weights.double()
    w = torch.where(place < live, w, 0.0)[:, :, None]
    out, size = (w * y).sum(1), (w * y).abs().sum(1)
    if residual is not None:
        out, size = out + residual.double(), size + residual.double().abs()
    return rounded(out, size * (place.shape[1] + 2) * E23, out_dtype)


def combine_backward(rows, place, live, weights, dout, dtype):
    at = place.long()
    ok = (place < live)[:, :, None]
    w = torch.ones(place.shape, dtype=torch.float64, device=rows.device) if weights is None else weights.double()
    d = torch.where(ok, w[:, :, None] * dout.double()[:, None], 0.0)
    drows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    drows[at.reshape(-1)] = d.view(-1, rows.shape[1])
    terms = torch.where(ok, rows.double()[at] * dout.double()[:, None], 0.0)
    # eight terms at a time in fp32, the rest in 64 bits
    return {"drows": rounded(drows, drows.abs() * E23, dtype), "dweights": (terms.sum(2), terms.abs().sum(2) * 12 * E23 + 1e-37)}



def _parts(parts):
    """Relative error of a product with a value held in bf16 parts: 8 bits each, rounded."""
    return 2.0 ** -(8 * parts + 1)


def adapters_forward(q, dtype, out_dtype):
    """{h, out} with bounds: h a sum of K products in fp32; out the sum of r products of h, held in fp32 or, beside bf16
    matrices, in two bf16 parts (three for an fp32 output)."""
    ids = q["ids"].long()
    n, r, K = q["down"].shape
    T, N = len(ids), q["up"].shape[1]
    h = torch.zeros(T, r, dtype=torch.float64, device=ids.device)
    eh, out, eout = h.clone(), torch.zeros(T, N, dtype=torch.float64, device=ids.device), torch.zeros(T, N, dtype=torch.float64, device=ids.device)
    split = _parts(3 if out_dtype is torch.float32 else 2) if dtype is torch.bfloat16 else 0
    for i in range(n):
        at = (ids == i).nonzero().view(-1)
        if not len(at):
            continue
        x, a, b, s = q["x"][at].double(), q["down"][i].double(), q["up"][i].double(), float(q["scale"][i])
        h[at] = x @ a.t()
        eh[at] = (x.abs() @ a.abs().t()) * ((K + 12) * E23)
        out[at] = s * (h[at] @ b.t())
        eout[at] = s * ((eh[at] + h[at].abs() * ((r + 8) * E23 + split)) @ b.abs().t())
    if q["residual"] is not None:
        out = out + q["residual"].double()
    return {"h": (h, eh), "out": rounded(out, eout + out.abs() * E23, out_dtype)}


def adapters_backward(q, dtype, gd):
    ids = q["ids"].long()
    n, r, K = q["down"].shape
    T, N = len(ids), q["up"].shape[1]
    dx, edx = torch.zeros(T, K, dtype=torch.float64, device=ids.device), torch.zeros(T, K, dtype=torch.float64, device=ids.device)
    da, db = torch.zeros(n, r, K, dtype=torch.float64, device=ids.device), torch.zeros(n, N, r, dtype=torch.float64, device=ids.device)
    eda, edb = torch.zeros_like(da), torch.zeros_like(db)
    bf = dtype is torch.bfloat16
    split_x = _parts(2) if bf else 0
    split_w = _parts(3 if gd is torch.float32 else 2) if bf else 0
    for i in range(n):
        at = (ids == i).nonzero().view(-1)
        if not len(at):
            continue
        x, a, b, s = q["x"][at].double(), q["down"][i].double(), q["up"][i].double(), float(q["scale"][i])
        dy, h = q["dout"][at].double(), q["h"][at].double()
        g = s * (dy @ b)
        # (an fp32 dout beside bf16 matrices is held in three parts)
        eg = s * (dy.abs() @ b.abs()) * ((N + 14) * E23 + (_parts(3) if bf else 0))
        dx[at] = g @ a
        edx[at] = (eg + g.abs() * ((r + 8) * E23 + split_x)) @ a.abs()
        da[i] = g.t() @ x
        eda[i] = (eg + g.abs() * ((len(at) + 8) * E23 + split_w)).t() @ x.abs()
        db[i] = s * (dy.t() @ h)
        edb[i] = s * (dy.abs().t() @ (h.abs() * ((len(at) + 9) * E23 + split_w)))
    if q["res_x"] is not None:
        dx = dx + q["res_x"].double()
    return {"dx": rounded(dx, edx + dx.abs() * E23, dtype), "ddown": rounded(da, eda, gd), "dup": rounded(db, edb, gd)}
