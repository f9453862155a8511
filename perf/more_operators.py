"""What is measured of the operators around the layer's matrix products: the root-mean-square norm with the
residual's addition (8-bit output with scales, backward pass), tokens sorted by expert and back with their gradients,
and low-rank adapters of many requests beside a shared projection with theirs.

`own` false: the plain form, elementary torch operations in 32 bits (64 next to the borders of 8-bit values) rounded
once at the end.  `own` true: the framework's kernels, through the calls that a user's program makes."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
MOST_BYTES = 1.7e9  # of the largest listed case


def _norm(name, op, t, d, dtype, res, out="y", save=False):
    """res: "none", or the residual stream's type ("same" as x, "f32"); out "mx": 8 bits with scales."""
    return {"name": name, "op": op, "t": t, "d": d, "dtype": dtype, "res": res, "out": out, "save": save}


def _route(name, op, t, d, k, e, dtype, x="same", out="same", pad=0.0, ids="i32"):
    """k choices of e experts a token; x "mx": 8-bit tokens; pad: the share of the batch that is padding, with no expert."""
    return {"name": name, "op": op, "t": t, "d": d, "k": k, "e": e, "dtype": dtype, "x": x, "out": out, "pad": pad, "ids": ids}


def _adapt(name, op, t, k, n, r, a, dtype, out="same"):
    """a adapters of rank r beside a projection k to n."""
    return {"name": name, "op": op, "t": t, "k": k, "n": n, "r": r, "a": a, "dtype": dtype, "out": out}


def listed():
    return [
        # the norm in front of the decode layer (d 4096, fp32 running sum): one token, latency counts
        _norm("norm_fwd_1tok", "norm_forward", 1, 4096, "bf16", "f32"),
        # ... of a long prompt, handed on in 8 bits
        _norm("norm_fwd_prefill_mx", "norm_forward", 8192, 4096, "bf16", "f32", out="mx"),
        # a ragged training batch of a model with an odd width, fp16 throughout
        _norm("norm_fwd_ragged_f16", "norm_forward", 1217, 2731, "f16", "same", save=True),
        # training on the prefill layer's tokens: gradients of the sum and of the weights
        _norm("norm_bwd_prefill", "norm_backward", 4096, 4096, "bf16", "f32"),
        # a decode batch through the layer's 256 experts, top-6: sort, tokens out, outputs back onto the fp32 sum
        _route("route_fwd_16tok", "route_forward", 16, 4096, 6, 256, "bf16", out="f32"),
        # ... the prefill layer's 4096 tokens
        _route("route_fwd_prefill", "route_forward", 4096, 4096, 6, 256, "bf16", out="f32"),
        # a padded batch in 8 bits on a model of odd width with 60 experts, top-4, ids as torch.topk gives them
        _route("route_fwd_padded_mx", "route_forward", 1217, 1000, 4, 60, "f16", x="mx", pad=0.2, ids="i64"),
        # training the top-8 layer on 8192 tokens: the largest
        _route("route_bwd_top8", "route_backward", 8192, 4096, 8, 256, "bf16"),
        # a decode batch of 16 requests, each with its own of 64 adapters, beside a 4096 x 4096 projection
        _adapt("adapt_fwd_16tok", "adapt_forward", 16, 4096, 4096, 16, 64, "bf16"),
        # prompts of several requests at once
        _adapt("adapt_fwd_prefill", "adapt_forward", 4096, 4096, 4096, 16, 8, "bf16"),
        # a small fp32 model of odd widths
        _adapt("adapt_fwd_ragged_f32", "adapt_forward", 777, 1330, 1999, 12, 5, "f32"),
        # training four adapters at once beside the I 2048 layer's down projection
        _adapt("adapt_bwd_down", "adapt_backward", 8192, 2048, 4096, 32, 4, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _spread(rng, lo, hi):
    """A whole number spread over its logarithm, a multiple of 64 half of the time."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.5:
        v = max(64, v // 64 * 64)
    return v


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "route_forward", "route_backward", "adapt_forward", "adapt_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    t = _log(rng, 1, 8192)
    if op.startswith("norm"):
        c = _norm("", op, t, _spread(rng, 64, 8192), dtype, rng.choice(["none", "same", "f32"]))
        if op == "norm_forward":
            c["out"], c["save"] = rng.choice(["y", "y", "mx"]), rng.random() < 0.5
    elif op.startswith("route"):
        e = _log(rng, 4, 512)
        c = _route("", op, t, _spread(rng, 64, 8192), min(e, rng.randint(1, 8)), e, dtype, out=rng.choice(["same", "f32"]),
                   pad=rng.choice([0.0, 0.0, 0.1, 0.3]), ids=rng.choice(["i32", "i64"]))
        if op == "route_forward":
            c["x"] = rng.choice(["same", "same", "mx"])
    else:
        r = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)])
        c = _adapt("", op, t, _spread(rng, 64, 8192), _spread(rng, 64, 8192), r, min(_log(rng, 1, 128), 2048 // r), dtype,
                   out=rng.choice(["same", "same", "f32"]))
    del c["name"]
    over = work(c)["bytes"] / MOST_BYTES
    if over > 1:
        c["t"] = max(1, int(c["t"] / over))
    return c


def _res_size(case):
    return 4 if case["res"] == "f32" else SIZE[case["dtype"]]


def work(case):
    e, t = SIZE[case["dtype"]], case["t"]
    if case["op"].startswith("norm"):
        td, rs = t * case["d"], _res_size(case)
        if case["op"] == "norm_forward":
            out = 1 + 1 / 32 if case["out"] == "mx" else e
            return {"bytes": td * (e + out + (2 * rs if case["res"] != "none" else 0)) + e * case["d"] + 4 * t * case["save"],
                    "flops": 5.0 * td}
        two = case["res"] != "none"  # the gradient that comes past the norm; the sum's and x's own are one where they have one type
        return {"bytes": td * (2 * e + rs + rs * two + (rs if two and rs != e else 0)) + 2 * e * case["d"] + 4 * t, "flops": 9.0 * td}
    o = 4 if case["out"] == "f32" else e
    if case["op"].startswith("route"):
        rows, d = t * case["k"], case["d"]
        if case["op"] == "route_forward":
            x = 1 + 1 / 32 if case["x"] == "mx" else e
            return {"bytes": t * d * (x + 2 * o) + 2 * rows * d * e + rows * (16 if case["ids"] == "i64" else 12),
                    "flops": 2.0 * rows * d}
        return {"bytes": t * d * (o + e) + 3 * rows * d * e + 12 * rows, "flops": 4.0 * rows * d}
    k, n, r, a = case["k"], case["n"], case["r"], case["a"]
    used = min(a, t) * r * (k + n)
    if case["op"] == "adapt_forward":
        return {"bytes": t * (k * e + 2 * n * o) + used * e, "flops": 2.0 * t * r * (k + n)}
    return {"bytes": t * (3 * k * e + n * o + 4 * r) + used * e + a * r * (k + n) * e, "flops": 4.0 * t * r * (k + n)}


# ---- inputs --------------------------------------------------------------------------

def _quantised(v):
    """(values in e4m3, E8M0 scales) of v [t, d] in 64 bits: groups of 32 columns, each over the smallest power of two
    that brings it within 448 (at least 2^-127)."""
    t, d = v.shape
    groups = (d + 31) // 32
    padded = torch.nn.functional.pad(v, (0, groups * 32 - d)).view(t, groups, 32)
    m, e = torch.frexp(padded.abs().amax(2))  # m 2^e, m in [0.5, 1); 448 is 0.875 2^9
    byte = torch.where(m > 0, torch.where(m <= 0.875, e - 9, e - 8) + 127, 0).clamp(0, 254)
    q = padded * torch.exp2(127 - byte.double())[:, :, None]
    return q.view(t, groups * 32)[:, :d].float().to(torch.float8_e4m3fn), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _expanded(q, scale):
    return q.float() * scale.float().repeat_interleave(32, dim=1)[:, : q.shape[1]]


def _inputs(case, seed):
    """The tensors of a case: activations, gradients of the loss's scale, weights of a trained net's, the choices of a
    router whose experts are not equally liked, adapters of requests."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, t = DTYPES[case["dtype"]], case["t"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {}
    if case["op"].startswith("norm"):
        d, rt = case["d"], torch.float32 if case["res"] == "f32" else dt
        s["weight"] = (1 + torch.randn(d, generator=g, device="cuda") * 0.1).to(dt)
        if case["op"] == "norm_forward":
            s["x"] = normal(t, d)
            s["residual"] = normal(t, d, std=3.0, dtype=rt) if case["res"] != "none" else None
            return s
        s["sum"] = normal(t, d, std=3.0, dtype=rt)
        s["rstd"] = (s["sum"].double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = normal(t, d, std=0.02)
        s["dsum"] = normal(t, d, std=0.02, dtype=rt) if case["res"] != "none" else None
        return s
    ot = torch.float32 if case["out"] == "f32" else dt
    if case["op"].startswith("route"):
        d, k, e = case["d"], case["k"], case["e"]
        liked = torch.randn(e, generator=g, device="cuda")
        top, ids = (torch.randn(t, e, generator=g, device="cuda") + liked).topk(k, dim=1)
        ids[t - int(t * case["pad"]):] = -1
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["gates"] = top.softmax(1)
        s["rows"] = normal(t * k, d)
        # what the experts had no row for, they have not written
        s["rows"][t * k - int(t * case["pad"]) * k:] = float("nan")
        if case["op"] == "route_forward":
            s["x"] = normal(t, d)
            if case["x"] == "mx":
                s["x"], s["x_scale"] = _quantised(s["x"].double())
            s["residual"] = normal(t, d, std=3.0, dtype=ot)
            return s
        s["dout"] = normal(t, d, std=0.02, dtype=ot)
        s["drows"] = normal(t * k, d, std=0.02)
        return s
    k, n, r, a = case["k"], case["n"], case["r"], case["a"]
    if t <= 64:  # a decode batch: a request each
        ids = torch.randint(0, a, (t,), generator=g, device="cuda")
    else:  # prompts of requests, one after the other; some without an adapter
        cuts = torch.randint(0, t, (2 * a,), generator=g, device="cuda").sort().values
        request = (torch.arange(t, device="cuda")[:, None] >= cuts).sum(1)
        ids = torch.randint(-1 if a > 1 else 0, a, (2 * a + 1,), generator=g, device="cuda")[request]
    s["ids"] = ids.to(torch.int32)
    s["x"] = normal(t, k)
    s["down"], s["up"] = normal(a, r, k, std=k ** -0.5), normal(a, n, r, std=r ** -0.5)
    s["scale"] = torch.rand(a, generator=g, device="cuda") + 0.5
    if case["op"] == "adapt_forward":
        s["residual"] = normal(t, n, dtype=ot)  # the shared projection's output
        return s
    s["h"] = _low(s, s["x"], s["down"]).sum(1)
    s["dout"] = normal(t, n, std=0.02, dtype=ot)
    s["dx"] = normal(t, k, std=0.02)  # the shared projection's own gradient of x
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if case["op"] == "route_backward":  # the forward pass's order is still there
        s.update(_sorted(s["ids"], case["e"]))
    if own:  # the objects a program holds
        from expert_cache_ffn_amd.layer import LowRankAdapters, RMSNorm, TokenSort
        if case["op"].startswith("norm"):
            rt = torch.float32 if case["res"] == "f32" else None
            s["norm"] = RMSNorm(s["weight"], eps=EPS, sum_dtype=rt)
        elif case["op"].startswith("adapt"):
            s["adapters"] = LowRankAdapters(s["down"], s["up"], s["scale"], out_dtype=torch.float32 if case["out"] == "f32" else None)
        if case["op"] == "route_backward":
            s["sort"] = TokenSort(s["ids"], case["e"])
        elif case["op"] == "adapt_backward":
            s["sort"] = TokenSort(s["ids"], case["a"])
    return s


# ---- the plain form ------------------------------------------------------------------

def _sorted(ids, e):
    """Choices in order of their experts, equal ones in their own order, those of no expert last."""
    keys = torch.where((ids >= 0) & (ids < e), ids, e).reshape(-1).long()
    order = torch.argsort(keys, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=order.device)
    counts = (keys[:, None] == torch.arange(e, device=keys.device)).sum(0)
    return {"counts": counts.int(), "order": order.int(), "place": place.view(ids.shape), "chosen": (keys < e).view(ids.shape)}


def _mask(ids, a):
    return (ids[:, None] == torch.arange(a, device=ids.device)).float()


def _low(s, v, m):
    """[t, adapters, rank]: v with each adapter's m, zeros where it is not the token's own."""
    a, r, k = m.shape
    return (v.float() @ m.float().reshape(a * r, k).t()).view(-1, a, r) * _mask(s["ids"], a)[:, :, None]


def _plain(s):
    case = s["case"]
    dt, op = DTYPES[case["dtype"]], case["op"]
    if op == "norm_forward":
        v = s["x"].float()
        if s["residual"] is not None:
            v = (v + s["residual"].float()).to(s["residual"].dtype)
        wide = v.double() if case["out"] == "mx" else v.float()
        rstd = torch.rsqrt((wide * wide).mean(1, keepdim=True) + EPS)
        y = wide * rstd * s["weight"].to(wide.dtype)
        out = list(_quantised(y)) if case["out"] == "mx" else [y.to(dt)]
        if s["residual"] is not None:
            out.append(v)
        return out + [rstd.view(-1).float()] if case["save"] else out
    if op == "norm_backward":
        v, dy, rstd = s["sum"].float(), s["dy"].float(), s["rstd"][:, None]
        hat, g = v * rstd, dy * s["weight"].float()
        ds = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        if s["dsum"] is not None:
            ds = ds + s["dsum"].float()
        out = [ds.to(dt), (dy * hat).sum(0).to(dt)]
        return out + [ds] if case["res"] == "f32" and case["dtype"] != "f32" else out
    if op == "route_forward":
        o = _sorted(s["ids"], case["e"])
        x = _expanded(s["x"], s["x_scale"]) if case["x"] == "mx" else s["x"].float()
        at, chosen = o["order"].long(), o["chosen"]
        rows = torch.where(chosen.view(-1)[at][:, None], x[at // case["k"]], 0.0).to(dt)
        back = torch.where(chosen[:, :, None], s["gates"][:, :, None] * s["rows"].float()[o["place"]], 0.0)
        out = s["residual"].float() + back.sum(1)
        return [o["counts"], o["order"], rows, out.to(s["residual"].dtype)]
    if op == "route_backward":
        dout, chosen = s["dout"].float(), s["chosen"][:, :, None]
        drows = torch.where(chosen, s["gates"][:, :, None] * dout[:, None], 0.0).to(dt)
        dgates = torch.where(chosen, s["rows"].float()[s["place"]] * dout[:, None], 0.0).sum(2)
        dx = torch.where(chosen, s["drows"].float()[s["place"]], 0.0).sum(1)
        return [drows.view(-1, case["d"])[s["order"].long()], dgates, dx.to(dt)]
    a, r = case["a"], case["r"]
    if op == "adapt_forward":
        h = _low(s, s["x"], s["down"]) * s["scale"][:, None]
        y = h.view(-1, a * r) @ s["up"].float().transpose(1, 2).reshape(a * r, case["n"])
        return (s["residual"].float() + y).to(s["residual"].dtype)
    dy, x = s["dout"].float(), s["x"].float()
    mask = (_mask(s["ids"], a) * s["scale"])[:, :, None]
    g = (dy @ s["up"].float().transpose(1, 2).reshape(a * r, case["n"]).t()).view(-1, a, r) * mask
    g = g.view(-1, a * r)
    dx = s["dx"].float() + g @ s["down"].float().reshape(a * r, case["k"])
    ddown = (g.t() @ x).view(a, r, case["k"])
    h = (s["h"][:, None, :] * mask).view(-1, a * r)
    dup = (h.t() @ dy).view(a, r, case["n"]).transpose(1, 2)
    return [dx.to(dt), ddown.to(dt), dup.to(dt).contiguous()]


# ---- the framework's calls ------------------------------------------------------------

def _kernels(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm_forward":
        o = s["norm"].forward(s["x"], residual=s["residual"], y=case["out"] == "y", mx=case["out"] == "mx", save=case["save"])
        out = [o.q, o.scale] if case["out"] == "mx" else [o.y]
        if s["residual"] is not None:
            out.append(o.sum)
        return out + [o.rstd] if case["save"] else out
    if op == "norm_backward":
        dx, ds, dw = s["norm"].backward(s["sum"], s["rstd"], s["dy"], dsum=s["dsum"])
        return [dx, dw, ds] if case["res"] == "f32" and case["dtype"] != "f32" else [dx, dw]
    if op == "route_forward":
        from expert_cache_ffn_amd.layer import TokenSort
        sort = TokenSort(s["ids"], case["e"])
        if case["x"] == "mx":
            rows = sort.dispatch(s["x"], scale=s["x_scale"], dtype=DTYPES[case["dtype"]])
        else:
            rows = sort.dispatch(s["x"])
        out = sort.combine(s["rows"], s["gates"], residual=s["residual"])
        return [sort.counts, sort.order, rows, out]
    if op == "route_backward":
        drows, dgates = s["sort"].combine_backward(s["rows"], s["gates"], s["dout"])
        return [drows, dgates, s["sort"].dispatch_backward(s["drows"])]
    if op == "adapt_forward":
        return s["adapters"].forward(s["x"], s["ids"], residual=s["residual"])
    return list(s["adapters"].backward(s["x"], s["sort"], s["h"], s["dout"], residual=s["dx"]))


def run(state):
    return _kernels(state) if own else _plain(state)


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    q, op, t = _inputs(case, seed), case["op"], case["t"]
    f = {k: v.double() for k, v in q.items() if v is not None and v.is_floating_point()}
    if op == "norm_forward":
        v = f["x"]
        if q["residual"] is not None:
            v = (v + f["residual"]).to(q["residual"].dtype).double()
        rms = torch.linalg.vector_norm(v, dim=1, keepdim=True) / math.sqrt(case["d"])
        inverse = 1 / torch.hypot(rms, torch.full_like(rms, math.sqrt(EPS)))
        y = v * inverse * f["weight"]
        out = [y]
        if case["out"] == "mx":
            parts = torch.split(y, 32, dim=1)
            power = torch.stack([torch.ceil(torch.log2(p.abs().amax(1) / 448)) for p in parts], 1).clamp_min(-127)
            out = [torch.cat([torch.ldexp(p, -power[:, i:i + 1]) for i, p in enumerate(parts)], 1), torch.exp2(power)]
        if q["residual"] is not None:
            out.append(v)
        return out + [inverse.view(-1)] if case["save"] else out
    if op == "norm_backward":
        # the derivative of v / rms(v) . w along each column, the inverse rms as it was kept
        along = torch.einsum("td,td,d->t", f["dy"], f["sum"], f["weight"]) * f["rstd"] ** 3 / case["d"]
        ds = f["dy"] * f["weight"] * f["rstd"][:, None] - f["sum"] * along[:, None]
        if q["dsum"] is not None:
            ds = ds + f["dsum"]
        dw = torch.mv((f["dy"] * f["sum"]).t(), f["rstd"])
        return [ds, dw, ds] if case["res"] == "f32" and case["dtype"] != "f32" else [ds, dw]
    if op.startswith("route"):
        d, k, e = case["d"], case["k"], case["e"]
        flat = q["ids"].reshape(-1).long()
        order = torch.cat([(flat == i).nonzero().view(-1) for i in range(e)] + [((flat < 0) | (flat >= e)).nonzero().view(-1)])
        live = int(((flat >= 0) & (flat < e)).sum())
        token = order[:live] // k
        if op == "route_forward":
            x = f["x"]
            if case["x"] == "mx":
                x = torch.cat([p * f["x_scale"][:, i:i + 1] for i, p in enumerate(torch.split(x, 32, dim=1))], 1)
            rows = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
            rows[:live] = x[token]
            out = f["residual"].index_add(0, token, f["rows"][:live] * f["gates"].view(-1)[order[:live], None])
            return [None, None, rows, out]
        drows = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
        drows[:live] = f["dout"][token] * f["gates"].view(-1)[order[:live], None]
        dgates = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dgates[order[:live]] = torch.linalg.vecdot(f["rows"][:live], f["dout"][token])
        dx = torch.zeros(t, d, dtype=torch.float64, device="cuda").index_add(0, token, f["drows"][:live])
        return [drows, dgates.view(t, k), dx]
    if op == "adapt_forward":
        y = f["residual"].clone()
        for i in range(case["a"]):
            at = (q["ids"] == i).nonzero().view(-1)
            y[at] += f["scale"][i] * torch.mm(torch.mm(f["x"][at], f["down"][i].t()), f["up"][i].t())
        return y
    dx, ddown, dup = f["dx"].clone(), torch.zeros_like(f["down"]), torch.zeros_like(f["up"])
    for i in range(case["a"]):
        at = (q["ids"] == i).nonzero().view(-1)
        dy = f["dout"][at] * f["scale"][i]
        g = torch.mm(dy, f["up"][i])
        dx[at] += torch.mm(g, f["down"][i])
        ddown[i], dup[i] = torch.mm(g.t(), f["x"][at]), torch.mm(dy.t(), f["h"][at])
    return [dx, ddown, dup]
