"""Torch-side conveniences over the C ABI: device memory, streams and argument
structs.  Nothing here computes any part of the layer; every step of the
forward pass runs in libecf's kernels (or its host expert threads)."""
from __future__ import annotations

import warnings
from functools import cached_property
from typing import NamedTuple

import torch

from . import _lib as L

_TORCH_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _ptr(t):
    return 0 if t is None else int(t.data_ptr())


def blob_sections(shape: L.Shape):
    """[(name, byte offset)] of one expert blob, in ecf_expert_layout order."""
    offs = L.ecf_expert_layout(shape)
    names = ["w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down"]
    n = 6 if shape.w_dtype == L.ECF_MXFP4 else 3
    return list(zip(names[:n], offs[:n]))


def pack_expert(shape: L.Shape, tensors: dict, blob: torch.Tensor):
    """Copy one expert's tensors into a uint8 blob view at the layout offsets."""
    for name, off in blob_sections(shape):
        t = tensors[name].contiguous()
        raw = t.view(torch.uint8).reshape(-1)
        blob[off:off + raw.numel()].copy_(raw)


class ExpertPool:
    """All experts of one layer resident in one device buffer [E, slot_bytes]."""

    def __init__(self, shape: L.Shape, device="cuda", n_experts=None):
        self.shape = shape
        self.slot_bytes = L.ecf_expert_bytes(shape)
        E = n_experts or shape.n_experts
        self.buf = torch.empty((E, self.slot_bytes), dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.ptrs = torch.tensor([base + e * self.slot_bytes for e in range(E)], dtype=torch.int64,
                                 device=device)

    def load(self, e: int, tensors: dict):
        pack_expert(self.shape, tensors, self.buf[e])


class Layer:
    """One MoE layer call site: owns its workspace and builds LayerArgs.

    LayerArgs carries raw device addresses only: every tensor passed to args()
    must stay referenced until the forward call's work has finished on the
    stream (a temporary such as `w.cuda()` would be freed, and its memory
    reused, while the kernels still read it)."""

    def __init__(self, shape: L.Shape, max_tokens: int, device="cuda"):
        self.shape = shape
        self.max_tokens = max_tokens
        self.ws_bytes = L.ecf_workspace_bytes(shape, max_tokens)
        self.ws = torch.empty(self.ws_bytes + 256, dtype=torch.uint8, device=device)
        base = self.ws.data_ptr()
        self.ws_ptr = (base + 255) & ~255
        self.device = device

    def args(self, *, layer=0, router_w=None, router_logits=None, expert_ptrs=None, cache=None,
             b_p=0.4, b_h=1.0, q_mode=L.ECF_Q_AUTO, q_fixed=0, path=L.ECF_PATH_AUTO, stream=None,
             copy_stream=None, residual=None, out_act=None, topk_idx=None, topk_gate=None, counts=None,
             perm=None, logits_out=None) -> L.LayerArgs:
        a = L.LayerArgs()
        a.shape = self.shape
        a.layer = layer
        a.d_router_w = _ptr(router_w) or None
        a.d_router_logits = _ptr(router_logits) or None
        a.d_expert_ptrs = _ptr(expert_ptrs) or None
        a.cache = cache or None
        a.b_p, a.b_h = float(b_p), float(b_h)
        a.q_mode, a.q_fixed, a.path = int(q_mode), int(q_fixed), int(path)
        a.d_ws = self.ws_ptr
        a.ws_bytes = self.ws_bytes
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        a.stream = st.cuda_stream or None
        a.copy_stream = (copy_stream.cuda_stream or None) if copy_stream is not None else None
        a.d_residual = _ptr(residual) or None
        a.d_out_act = _ptr(out_act) or None
        a.d_topk_idx = _ptr(topk_idx) or None
        a.d_topk_gate = _ptr(topk_gate) or None
        a.d_counts = _ptr(counts) or None
        a.d_perm = _ptr(perm) or None
        a.d_logits = _ptr(logits_out) or None
        return a

    def forward(self, args: L.LayerArgs, x: torch.Tensor, out: torch.Tensor, want_stats=True):
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens > workspace capacity {self.max_tokens}")
        assert x.is_contiguous() and out.is_contiguous() and out.dtype == torch.float32
        return L.moe_layer_forward(args, x.data_ptr(), T, out.data_ptr(), want_stats)


# ---- dense feed-forward operators -------------------------------------------------

# The address of a device's current stream.  torch.cuda.current_stream() builds a
# Stream object around it, 2.8 us of the 11 a one-token call took on the host.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice

_DENSE_DT = {torch.float32: L.ECF_F32, torch.bfloat16: L.ECF_BF16, torch.float16: L.ECF_F16}


def _dense_dt(dtype, what):
    if dtype not in _DENSE_DT:
        raise ValueError(f"{what} must be float32, bfloat16 or float16, got {dtype}")
    return _DENSE_DT[dtype]


def _matrix(name, t, rows, cols, dtype, device):
    """(address, row stride) of a [rows, cols] operand; its rows may lie apart but not overlap."""
    if not isinstance(t, torch.Tensor) or t.shape != (rows, cols):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor, got {tuple(getattr(t, 'shape', ()))}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weights are on {device}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows (strides {t.stride()})")
    if rows <= 1:
        ld = cols  # a single row's stride says nothing
    elif ld < cols:
        raise ValueError(f"the rows of {name} overlap (strides {t.stride()}): make it contiguous")
    return t.data_ptr(), ld


def _vector(name, t, n, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.shape != (n,) or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be a [{n}] tensor of {dtype} on {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _kept(*tensors):
    """The tensors' own views of their memory: it stays theirs if w.data is replaced."""
    return [None if t is None else t.detach() for t in tensors]


def _warn_untracked(what, call="backward"):
    """A forward call that something requires gradients of; it gives none where they are on."""
    if torch.is_grad_enabled():
        name = what if "." in what else f"{what}.forward"
        warnings.warn(f"{name} is outside autograd: its output has no gradient function although the weights or "
                      f"an input require gradients.  Run it under torch.no_grad(), and call {call}() with the "
                      "output's gradient", stacklevel=3)


class _Dense:
    """What the two operators share: the weights' checks, workspaces and streams.

    They are outside autograd: outputs never carry a gradient function, and a training
    step calls backward() itself, best under torch.no_grad().  forward() warns where
    gradients are on, the weights or an input require them and nothing is saved for
    backward().

    A call runs on the current stream of the weights' device and takes its
    workspace from torch's allocator for that stream, so calls on several
    streams, and captured graphs, never share one."""

    def _setup(self, w, act, what):
        if not isinstance(w, torch.Tensor) or w.dim() != 2 or not w.is_cuda or 0 in w.shape:
            raise ValueError(f"{what} must be a non-empty 2-D tensor on the GPU")
        if act not in L.ACTS:
            raise ValueError(f"act must be one of {sorted(L.ACTS)}, got {act!r}")
        self.device, self.dtype, self.act = w.device, w.dtype, act
        self._dt = _dense_dt(w.dtype, what)
        # torch.empty of each type a call makes, its device looked up once (1.4 -> 1.1 us)
        self._empty = {dt: torch.empty(0, dtype=dt, device=w.device).new_empty
                       for dt in (w.dtype, torch.float32, torch.uint8)}
        self._ws_of = {}

    def _tokens(self, x):
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a 2-D tensor [tokens, features]")
        return x.shape[0]

    def _run(self, fn, a, T, backward):
        if _current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._run(fn, a, T, backward)
        n = self._ws_of.get((T, backward))
        if n is None:
            n = self._ws_bytes(T, backward)
            if len(self._ws_of) > 4096:
                self._ws_of.clear()
            self._ws_of[T, backward] = n
        if n:
            ws = self._empty[torch.uint8](n)
            a.d_ws, a.ws_bytes = ws.data_ptr(), n
        a.stream = _raw_stream(self.device.index) or None
        fn(a, T)

    def _wgrad(self, w_grad_dtype):
        dt = self.dtype if w_grad_dtype is None else w_grad_dtype
        if dt is not self.dtype and dt is not torch.float32:
            raise ValueError(f"w_grad_dtype must be {self.dtype} or torch.float32, got {dt}")
        return dt

    def _out(self, name, t, rows, cols, dtype):
        if t is None:
            t = self._empty[dtype]((rows, cols))
            return t, t.data_ptr(), cols
        return (t,) + _matrix(name, t, rows, cols, dtype, self.device)


class GatedProjection(_Dense):
    """h = act(x W_gate^T + b_gate) * (x W_up^T + b_up): the first half of a gated
    feed-forward block (SwiGLU with act "silu"), in one kernel.

    w_gate, w_up [inter, hidden] in fp32, bf16 or fp16, with the same row stride;
    b_gate, b_up [inter] or None.  The object keeps their memory: in-place updates of
    the weights are seen by the next call, a tensor given other memory (w.data = ...)
    needs a new object."""

    def __init__(self, w_gate, w_up, b_gate=None, b_up=None, act="silu"):
        self._setup(w_gate, act, "w_gate")
        self.inter, self.hidden = w_gate.shape
        a = L.GatedArgs()
        a.hidden, a.inter, a.dtype, a.act = self.hidden, self.inter, self._dt, L.ACTS[act]
        a.d_w_gate, a.ld_w = _matrix("w_gate", w_gate, self.inter, self.hidden, self.dtype, self.device)
        a.d_w_up, ld = _matrix("w_up", w_up, self.inter, self.hidden, self.dtype, self.device)
        if ld != a.ld_w:
            raise ValueError(f"w_gate and w_up must have the same row stride ({a.ld_w} and {ld})")
        a.d_b_gate = _vector("b_gate", b_gate, self.inter, self.dtype, self.device)
        a.d_b_up = _vector("b_up", b_up, self.inter, self.dtype, self.device)
        self._learns = any(t is not None and t.requires_grad for t in (w_gate, w_up, b_gate, b_up))
        self.w_gate, self.w_up, self.b_gate, self.b_up = _kept(w_gate, w_up, b_gate, b_up)
        self._a = a

    def _ws_bytes(self, T, backward):
        return L.ecf_gated_workspace_bytes(self.hidden, self.inter, self._dt, T, backward)

    def forward(self, x, out=None, save=False):
        """h [T, inter] (into `out` if given); with save, (h, a, b): also the two
        sums, rounded to the weights' type, for backward()."""
        T = self._tokens(x)
        a = L.GatedArgs.from_buffer_copy(self._a)
        a.d_x, a.ld_x = _matrix("x", x, T, self.hidden, self.dtype, self.device)
        if (self._learns or x.requires_grad) and not save:
            _warn_untracked("GatedProjection")
        h, a.d_h, a.ld_h = self._out("out", out, T, self.inter, self.dtype)
        if save:
            sa, a.d_a, a.ld_ab = self._out("a", None, T, self.inter, self.dtype)
            sb, a.d_b, _ = self._out("b", None, T, self.inter, self.dtype)
        self._run(L.ecf_gated_forward, a, T, 0)
        return (h, sa, sb) if save else h

    def backward(self, x, a, b, dh, w_grad_dtype=None, dx=None, need_dx=True, need_dw=True):
        """(dx, dw_gate, dw_up, db_gate, db_up) for the gradient dh of h, from the x
        of the forward call and the a and b it saved; the last two are None without
        the biases, dx without need_dx (the network's first layer), the other four
        without need_dw (frozen weights).  Weight and bias gradients come in
        w_grad_dtype (the weights' type, or torch.float32)."""
        T, gd = self._tokens(x), self._wgrad(w_grad_dtype)
        q = L.GatedArgs.from_buffer_copy(self._a)
        q.wgrad_dtype = _DENSE_DT[gd]
        q.d_x, q.ld_x = _matrix("x", x, T, self.hidden, self.dtype, self.device)
        q.d_a, q.ld_ab = _matrix("a", a, T, self.inter, self.dtype, self.device)
        q.d_b, ld = _matrix("b", b, T, self.inter, self.dtype, self.device)
        if ld != q.ld_ab:
            raise ValueError(f"a and b must have the same row stride ({q.ld_ab} and {ld})")
        q.d_dh, q.ld_dh = _matrix("dh", dh, T, self.inter, self.dtype, self.device)
        dwg = dwu = dbg = dbu = None
        if need_dx:
            dx, q.d_dx, q.ld_dx = self._out("dx", dx, T, self.hidden, self.dtype)
        elif dx is not None:
            raise ValueError("dx is given but need_dx is false")
        if need_dw:
            dwg, q.d_dw_gate, q.ld_dw = self._out("dw_gate", None, self.inter, self.hidden, gd)
            dwu, q.d_dw_up, _ = self._out("dw_up", None, self.inter, self.hidden, gd)
            if self.b_gate is not None:
                dbg = self._empty[gd](self.inter)
                q.d_db_gate = dbg.data_ptr()
            if self.b_up is not None:
                dbu = self._empty[gd](self.inter)
                q.d_db_up = dbu.data_ptr()
        self._run(L.ecf_gated_backward, q, T, 1)
        return dx, dwg, dwu, dbg, dbu


class Linear(_Dense):
    """y = act(x W^T + bias) + residual, with bias, activation and residual in the
    product's epilogue.

    w [out_features, in_features] in fp32, bf16 or fp16, bias [out_features] or None
    (kept as GatedProjection keeps its weights).
    y, the residual and dy are of out_dtype: the weights' type, or torch.float32 (the
    running sum a moe_layer_forward call takes as its residual)."""

    def __init__(self, w, bias=None, act="none", out_dtype=None):
        self._setup(w, act, "w")
        self.out_features, self.in_features = w.shape
        self.out_dtype = w.dtype if out_dtype is None else out_dtype
        if self.out_dtype is not w.dtype and self.out_dtype is not torch.float32:
            raise ValueError(f"out_dtype must be {w.dtype} or torch.float32, got {out_dtype}")
        a = L.LinearArgs()
        a.in_features, a.out_features, a.dtype, a.act = self.in_features, self.out_features, self._dt, L.ACTS[act]
        a.out_dtype = _DENSE_DT[self.out_dtype]
        a.d_w, a.ld_w = _matrix("w", w, self.out_features, self.in_features, self.dtype, self.device)
        a.d_bias = _vector("bias", bias, self.out_features, self.dtype, self.device)
        # how the backward pass's workspace is asked for: 2, dy goes into its products as it is
        self._back = 2 if act == "none" and self.out_dtype is w.dtype else 1
        self._learns = w.requires_grad or (bias is not None and bias.requires_grad)
        self.w, self.bias = _kept(w, bias)
        self._a = a

    def _ws_bytes(self, T, backward):
        return L.ecf_linear_workspace_bytes(self.in_features, self.out_features, self._dt, T, backward)

    def forward(self, x, residual=None, out=None, save=False):
        """y [T, out_features] (into `out` if given, which may be the residual); with
        save, (y, z): also z = x W^T + bias, rounded to the weights' type, for
        backward() through an activation."""
        T = self._tokens(x)
        a = L.LinearArgs.from_buffer_copy(self._a)
        a.d_x, a.ld_x = _matrix("x", x, T, self.in_features, self.dtype, self.device)
        if residual is not None:
            a.d_residual, a.ld_residual = _matrix("residual", residual, T, self.out_features, self.out_dtype,
                                                  self.device)
        if (self._learns or x.requires_grad or residual is not None and residual.requires_grad) and not save:
            _warn_untracked("Linear")
        y, a.d_out, a.ld_out = self._out("out", out, T, self.out_features, self.out_dtype)
        if save:
            z, a.d_z, a.ld_z = self._out("z", None, T, self.out_features, self.dtype)
        self._run(L.ecf_linear_forward, a, T, 0)
        return (y, z) if save else y

    def backward(self, x, dout, z=None, w_grad_dtype=None, dx=None, need_dx=True, need_dw=True):
        """(dx, dw, dbias) for the gradient dout of y, from the x of the forward call
        and, with an activation, the z it saved; dbias is None without a bias, dx
        without need_dx, the other two without need_dw.  The residual's gradient is
        dout itself."""
        T, gd = self._tokens(x), self._wgrad(w_grad_dtype)
        q = L.LinearArgs.from_buffer_copy(self._a)
        q.wgrad_dtype = _DENSE_DT[gd]
        q.d_x, q.ld_x = _matrix("x", x, T, self.in_features, self.dtype, self.device)
        if self.act != "none":
            q.d_z, q.ld_z = _matrix("z", z, T, self.out_features, self.dtype, self.device)
        q.d_dout, q.ld_dout = _matrix("dout", dout, T, self.out_features, self.out_dtype, self.device)
        dw = db = None
        if need_dx:
            dx, q.d_dx, q.ld_dx = self._out("dx", dx, T, self.in_features, self.dtype)
        elif dx is not None:
            raise ValueError("dx is given but need_dx is false")
        if need_dw:
            dw, q.d_dw, q.ld_dw = self._out("dw", None, self.out_features, self.in_features, gd)
            if self.bias is not None:
                db = self._empty[gd](self.out_features)
                q.d_dbias = db.data_ptr()
        self._run(L.ecf_linear_backward, q, T, self._back)
        return dx, dw, db


# ---- token operators ------------------------------------------------------------------

class NormOut(NamedTuple):
    """What RMSNorm.forward gives; None for what was not asked for."""
    y: torch.Tensor | None
    sum: torch.Tensor
    rstd: torch.Tensor | None
    q: torch.Tensor | None
    scale: torch.Tensor | None


_EMPTY = {}  # torch.empty of each type a call makes, by device


class _Tokens:
    """What the token operators share: workspaces and streams.  A call runs on the current
    stream of the operator's device and takes its workspace and outputs from torch's
    allocator for that stream, so calls on several streams, and captured graphs, never
    share one.  As the dense operators they are outside autograd."""

    def _setup(self, device):
        self.device = device
        if device not in _EMPTY:
            _EMPTY[device] = {dt: torch.empty(0, dtype=dt, device=device).new_empty
                              for dt in (torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8,
                                         torch.float8_e4m3fn, torch.float8_e8m0fnu)}
        self._empty = _EMPTY[device]

    def _run(self, fn, a, T, ws_bytes=0):
        if _current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._run(fn, a, T, ws_bytes)
        if ws_bytes:
            ws = self._empty[torch.uint8](ws_bytes)
            a.d_ws, a.ws_bytes = ws.data_ptr(), ws_bytes
        a.stream = _raw_stream(self.device.index) or None
        fn(a, T)

    def _out(self, name, t, rows, cols, dtype):
        if t is None:
            t = self._empty[dtype]((rows, cols))
            return t, t.data_ptr(), cols
        return (t,) + _matrix(name, t, rows, cols, dtype, self.device)

    def _matrix_of(self, name, t, what="tokens"):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D tensor [{what}, features]")
        return t.shape[0]


def _ws_cached(cache, key, size):
    n = cache.get(key)
    if n is None:
        if len(cache) > 4096:
            cache.clear()
        n = cache[key] = size(*key)
    return n


class RMSNorm(_Tokens):
    """y = sum * rstd * weight with sum = x + residual and rstd = 1 / sqrt(mean(sum^2) + eps).

    weight [hidden] in `dtype` or fp32; dtype (the weight's unless given) is the type of x,
    y and their gradients, sum_dtype (dtype unless given, or torch.float32) that of the
    residual, the sum and their gradients: the sum a moe_layer_forward call takes as its
    residual is fp32.  The object keeps the weight's memory, as GatedProjection does."""

    def __init__(self, weight, eps=1e-6, dtype=None, sum_dtype=None):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 1 or not weight.is_cuda or 0 in weight.shape:
            raise ValueError("weight must be a non-empty 1-D tensor on the GPU")
        self._setup(weight.device)
        self.hidden, = weight.shape
        self.dtype = weight.dtype if dtype is None else dtype
        self.sum_dtype = self.dtype if sum_dtype is None else sum_dtype
        for name, t in (("weight", weight.dtype), ("sum_dtype", self.sum_dtype)):
            if t is not self.dtype and t is not torch.float32:
                raise ValueError(f"{name} must be {self.dtype} or torch.float32, got {t}")
        a = L.NormArgs()
        a.hidden, a.eps = self.hidden, float(eps)
        a.dtype, a.sum_dtype = _dense_dt(self.dtype, "dtype"), _DENSE_DT[self.sum_dtype]
        a.weight_dtype = a.wgrad_dtype = _DENSE_DT[weight.dtype]
        a.d_weight = _vector("weight", weight, self.hidden, weight.dtype, self.device)
        if not 0 <= float(eps) < float("inf"):
            raise ValueError(f"eps must be finite and not negative, got {eps}")
        self._learns = weight.requires_grad
        self.weight, = _kept(weight)
        self._a = a
        self._ws_of = {}

    def forward(self, x, residual=None, y=True, mx=False, save=False, out=None, sum_out=None):
        """NormOut(y, sum, rstd, q, scale): y (into `out` if given); the sum (into sum_out if
        given, which may be the residual; x itself without a residual); with save, rstd for
        backward(); with mx, y in 8 bits: q [T, hidden] of torch.float8_e4m3fn and scale
        [T, ceil(hidden / 32)] of torch.float8_e8m0fnu, y then only with y=True too."""
        T = self._matrix_of("x", x)
        a = L.NormArgs.from_buffer_copy(self._a)
        a.d_x, a.ld_x = _matrix("x", x, T, self.hidden, self.dtype, self.device)
        if (self._learns or x.requires_grad or residual is not None and residual.requires_grad) and not save:
            _warn_untracked("RMSNorm")
        total, o, rstd, q, scale = x, None, None, None, None
        if residual is not None:
            a.d_residual, a.ld_residual = _matrix("residual", residual, T, self.hidden, self.sum_dtype, self.device)
            total, a.d_sum, a.ld_sum = self._out("sum_out", sum_out, T, self.hidden, self.sum_dtype)
        elif sum_out is not None:
            raise ValueError("sum_out is given without a residual: the sum is x")
        if y:
            o, a.d_y, a.ld_y = self._out("out", out, T, self.hidden, self.dtype)
        elif out is not None or not mx:
            raise ValueError("y=False needs mx=True and no out")
        if mx:
            q, a.d_q, _ = self._out("q", None, T, self.hidden, torch.float8_e4m3fn)
            scale, a.d_q_scale, _ = self._out("scale", None, T, (self.hidden + 31) // 32, torch.float8_e8m0fnu)
        if save:
            rstd = self._empty[torch.float32](T)
            a.d_rstd = rstd.data_ptr()
        self._run(L.ecf_norm_forward, a, T)
        return NormOut(o, total, rstd, q, scale)

    def backward(self, total, rstd, dy, dsum=None, w_grad_dtype=None, ds=None, need_dx=True, need_dw=True):
        """(dx, ds, dweight) for the gradient dy of y and dsum of the sum (what reaches it past
        the norm, or None), from the sum and rstd of the forward call.  ds (into `ds` if given,
        which may be dsum) is the gradient of the residual, dx the same values in x's type: one
        tensor where the types are one.  dx and ds are None without need_dx, dweight
        without need_dw; it comes in w_grad_dtype (the weight's type, or torch.float32)."""
        T = self._matrix_of("total", total)
        a = L.NormArgs.from_buffer_copy(self._a)
        gd = self.weight.dtype if w_grad_dtype is None else w_grad_dtype
        if gd is not self.weight.dtype and gd is not torch.float32:
            raise ValueError(f"w_grad_dtype must be {self.weight.dtype} or torch.float32, got {gd}")
        a.wgrad_dtype = _DENSE_DT[gd]
        st = total.dtype  # (a norm without a residual has x for its sum)
        if st is not self.dtype and st is not self.sum_dtype:
            raise ValueError(f"total must be {self.sum_dtype} (or {self.dtype}, an x without a residual), got {st}")
        a.sum_dtype = _DENSE_DT[st]
        a.d_sum, a.ld_sum = _matrix("total", total, T, self.hidden, st, self.device)
        a.d_rstd = _vector("rstd", rstd, T, torch.float32, self.device)
        if a.d_rstd is None and T:
            raise ValueError("rstd is missing: forward(save=True) gives it")
        a.d_dy, a.ld_dy = _matrix("dy", dy, T, self.hidden, self.dtype, self.device)
        if dsum is not None:
            a.d_dsum, a.ld_dsum = _matrix("dsum", dsum, T, self.hidden, st, self.device)
        dx = dw = None
        if need_dx:
            ds, a.d_ds, a.ld_ds = self._out("ds", ds, T, self.hidden, st)
            if st is self.dtype:
                dx = ds
            else:
                dx, a.d_dx, a.ld_dx = self._out("dx", None, T, self.hidden, self.dtype)
        elif ds is not None:
            raise ValueError("ds is given but need_dx is false")
        n = 0
        if need_dw:
            dw = self._empty[gd](self.hidden)
            a.d_dweight = dw.data_ptr()
            n = _ws_cached(self._ws_of, (self.hidden, T, 1), L.ecf_norm_workspace_bytes)
        self._run(L.ecf_norm_backward, a, T, n)
        return dx, ds, dw


_SORT_WS = {}  # bytes by (experts, k, tokens)


class TokenSort(_Tokens):
    """The choices of tokens in the order of their experts: ids [T, k] (or [T], k = 1) of
    torch.int32 or torch.int64, the choice f = t * k + j of token t.  A choice outside
    [0, n_experts) is of no expert and comes last.

    counts [n_experts], offsets [n_experts + 1] (the rows of expert e are offsets[e] to
    offsets[e + 1]), order [T * k] (row -> f), place [T, k] (f -> row) and tiles
    [n_experts + 2] (first tile of 64 rows of each expert) are int32 tensors on the ids'
    device, made by the constructor's call on the current stream.  The experts between
    dispatch() and combine() are the caller's: GatedProjection and Linear over the
    rows of each.  The tables belong to the stream that made them, as any tensor of torch's
    allocator: where work on another stream reads them, keep the object until it is done.
    ids are read again by LowRankAdapters: they stay as they are while the object is used."""

    def __init__(self, ids, n_experts):
        if not isinstance(ids, torch.Tensor) or ids.dim() not in (1, 2) or not ids.is_cuda:
            raise ValueError("ids must be a [tokens, k] or [tokens] tensor on the GPU")
        if ids.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
        self._setup(ids.device)
        self.ids, = _kept(ids)
        self.tokens, self.top_k = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
        self.n_experts = int(n_experts)
        wide = ids if ids.dim() == 2 else ids.unsqueeze(1)
        a = L.SortArgs()
        a.n_experts, a.top_k, a.idx_bytes = self.n_experts, self.top_k, ids.element_size()
        a.d_idx, a.ld_idx = _matrix("ids", wide, self.tokens, self.top_k, ids.dtype, self.device)
        n_ws = _ws_cached(_SORT_WS, (self.n_experts, self.top_k, self.tokens), L.ecf_token_sort_workspace_bytes)
        E, R = self.n_experts, self.tokens * self.top_k
        # one allocation: offsets, counts, tiles, order, place, each at a 16-byte boundary
        e4, r4 = (E + 5) // 4 * 4, (R + 3) // 4 * 4
        self._buf = self._empty[torch.int32](3 * e4 + 2 * r4)
        p = self._buf.data_ptr()
        a.d_offsets, a.d_counts, a.d_tiles, a.d_order, a.d_place = p, p + 4 * e4, p + 8 * e4, p + 12 * e4, p + 12 * e4 + 4 * r4
        self._run(L.ecf_token_sort, a, self.tokens, n_ws)
        t = self._a = L.TokenArgs()
        t.n_experts, t.top_k, t.d_offsets, t.d_place = E, self.top_k, p, a.d_place
        self._s = a

    def _part(self, address, n):
        at = (address - self._s.d_offsets) // 4
        return self._buf[at:at + n]

    # (views of one buffer, made when asked for: each costs the host as much as a launch)
    @cached_property
    def counts(self):
        return self._part(self._s.d_counts, self.n_experts)

    @cached_property
    def offsets(self):
        return self._part(self._s.d_offsets, self.n_experts + 1)

    @cached_property
    def tiles(self):
        return self._part(self._s.d_tiles, self.n_experts + 2)

    @cached_property
    def order(self):
        return self._part(self._s.d_order, self.tokens * self.top_k)

    @cached_property
    def place(self):
        return self._part(self._s.d_place, self.tokens * self.top_k).view(self.tokens, self.top_k)

    def _weights(self, w):
        if not isinstance(w, torch.Tensor) or w.shape != (self.tokens, self.top_k) or w.dtype is not torch.float32 \
                or w.device != self.device or not w.is_contiguous():
            raise ValueError(f"weights must be a contiguous float32 tensor [{self.tokens}, {self.top_k}] on {self.device}")
        return w.data_ptr()

    def _args(self, t, rows, name):
        n = self._matrix_of(name, t)
        if n != rows:
            raise ValueError(f"{name} must have {rows} rows, got {n}")
        a = L.TokenArgs.from_buffer_copy(self._a)
        a.hidden = t.shape[1]
        return a, t.shape[1]

    def dispatch(self, x, scale=None, dtype=None, out=None):
        """rows [T * k, d]: rows[place[t, j]] = x[t], zeros behind the last expert's rows.  With a
        scale, x is 8-bit (RMSNorm.forward's q and scale) and the rows are of `dtype`."""
        a, d = self._args(x, self.tokens, "x")
        if scale is None:
            if dtype is not None and dtype is not x.dtype:
                raise ValueError(f"the rows have x's type {x.dtype}, got {dtype}")
            dtype = x.dtype
            a.dtype = a.token_dtype = _dense_dt(dtype, "x")
            a.d_x, a.ld_x = _matrix("x", x, self.tokens, d, dtype, self.device)
            if x.requires_grad:
                _warn_untracked("TokenSort.dispatch", call="dispatch_backward")
        else:
            a.dtype, a.token_dtype = _dense_dt(dtype, "dtype"), L.ECF_MXFP8
            a.d_x, a.ld_x = _matrix("x", x, self.tokens, d, torch.float8_e4m3fn, self.device)
            a.d_x_scale, a.ld_x_scale = _matrix("scale", scale, self.tokens, (d + 31) // 32, torch.float8_e8m0fnu, self.device)
        rows, a.d_rows, a.ld_rows = self._out("out", out, self.tokens * self.top_k, d, dtype)
        self._run(L.ecf_token_dispatch, a, self.tokens)
        return rows

    def combine(self, rows, weights=None, residual=None, out=None, out_dtype=None):
        """out [T, d] = residual[t] + sum_j weights[t, j] * rows[place[t, j]] over the choices of an
        expert (into `out` if given, which may be the residual); of the residual's or out_dtype's
        type, else the rows' (the rows' type or torch.float32)."""
        a, d = self._args(rows, self.tokens * self.top_k, "rows")
        a.dtype = _dense_dt(rows.dtype, "rows")
        a.d_rows, a.ld_rows = _matrix("rows", rows, self.tokens * self.top_k, d, rows.dtype, self.device)
        od = out_dtype if out_dtype is not None else out.dtype if out is not None \
            else residual.dtype if residual is not None else rows.dtype
        if od is not rows.dtype and od is not torch.float32:
            raise ValueError(f"out_dtype must be {rows.dtype} or torch.float32, got {od}")
        a.token_dtype = _DENSE_DT[od]
        if weights is not None:
            a.d_weight = self._weights(weights)
        if residual is not None:
            a.d_residual, a.ld_residual = _matrix("residual", residual, self.tokens, d, od, self.device)
        if rows.requires_grad or weights is not None and weights.requires_grad or residual is not None and residual.requires_grad:
            _warn_untracked("TokenSort.combine", call="combine_backward")
        out, a.d_out, a.ld_out = self._out("out", out, self.tokens, d, od)
        self._run(L.ecf_token_combine, a, self.tokens)
        return out

    def combine_backward(self, rows, weights, dout, need_drows=True, need_dweights=True):
        """(drows, dweights) for the gradient dout of combine()'s output: drows [T * k, d] in
        the rows' type, zeros behind the last expert's; dweights [T, k] in fp32, 0 for a choice of
        no expert, None without need_dweights or weights.  The residual's gradient is dout itself."""
        a, d = self._args(rows, self.tokens * self.top_k, "rows")
        a.dtype = _dense_dt(rows.dtype, "rows")
        a.d_rows, a.ld_rows = _matrix("rows", rows, self.tokens * self.top_k, d, rows.dtype, self.device)
        if not isinstance(dout, torch.Tensor) or dout.dtype is not rows.dtype and dout.dtype is not torch.float32:
            raise ValueError(f"dout must be a tensor of {rows.dtype} or torch.float32")
        a.token_dtype = _DENSE_DT[dout.dtype]
        a.d_dout, a.ld_dout = _matrix("dout", dout, self.tokens, d, dout.dtype, self.device)
        drows = dweights = None
        if weights is not None:
            a.d_weight = self._weights(weights)
            if need_dweights:
                dweights, a.d_dweight, _ = self._out("dweights", None, self.tokens, self.top_k, torch.float32)
        if need_drows:
            drows, a.d_drows, a.ld_drows = self._out("drows", None, self.tokens * self.top_k, d, rows.dtype)
        self._run(L.ecf_token_combine_backward, a, self.tokens)
        return drows, dweights

    def dispatch_backward(self, drows, residual=None, out=None):
        """dx [T, d] = residual[t] (a gradient that x has already, or None) + the sum of its rows' gradients."""
        return self.combine(drows, residual=residual, out=out)


class LowRankAdapters(_Tokens):
    """out[t] = residual[t] + scale[a] * up[a] (down[a] x[t]), a = ids[t]: low-rank adapters of
    many requests beside a shared projection, whose output is the residual (or Linear.forward
    takes this output as its residual).  A token whose id lies outside the stack has none.

    down [n, rank, in_features] and up [n, out_features, rank] in fp32, bf16 or fp16, of one rank
    (smaller ones are padded with zeros); scale [n] in fp32 or None (ones), a constant without a
    gradient; the residual, out and dout are of out_dtype: the weights' type, or torch.float32.
    ids: [T] of torch.int32 or torch.int64, or a TokenSort over them, which a step makes once for
    all its layers (the ids then stay as they are).  The object keeps the weights' memory, as
    Linear does."""

    def __init__(self, down, up, scale=None, out_dtype=None):
        if not isinstance(down, torch.Tensor) or down.dim() != 3 or not down.is_cuda or 0 in down.shape:
            raise ValueError("down must be a non-empty tensor [adapters, rank, in_features] on the GPU")
        self._setup(down.device)
        self.dtype = down.dtype
        self.n, self.rank, self.in_features = down.shape
        if not isinstance(up, torch.Tensor) or up.dim() != 3 or 0 in up.shape or up.shape[0] != self.n or up.shape[2] != self.rank:
            raise ValueError(f"up must be a non-empty tensor [{self.n}, out_features, {self.rank}]")
        self.out_features = up.shape[1]
        for name, t in (("down", down), ("up", up)):
            if t.dtype is not self.dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous tensor of {self.dtype} on {self.device}")
        self.out_dtype = self.dtype if out_dtype is None else out_dtype
        if self.out_dtype is not self.dtype and self.out_dtype is not torch.float32:
            raise ValueError(f"out_dtype must be {self.dtype} or torch.float32, got {out_dtype}")
        a = L.AdapterArgs()
        a.in_features, a.out_features, a.rank, a.n_adapters = self.in_features, self.out_features, self.rank, self.n
        a.dtype, a.out_dtype = _dense_dt(self.dtype, "down"), _DENSE_DT[self.out_dtype]
        a.d_a, a.d_b = down.data_ptr(), up.data_ptr()
        a.d_scale = _vector("scale", scale, self.n, torch.float32, self.device)
        if scale is not None and scale.requires_grad:
            raise ValueError("scale is a constant, backward() has no gradient for it: give scale.detach()")
        self._learns = down.requires_grad or up.requires_grad
        self.down, self.up, self.scale = _kept(down, up, scale)
        self._a = a
        self._ws_of = {}
        self._ws(0, 0)  # refuses a shape that no call takes

    def _ids(self, a, ids, T):
        """The ids as the call reads them, which the caller of this holds over the call."""
        if isinstance(ids, TokenSort):
            if (ids.tokens, ids.top_k, ids.n_experts) != (T, 1, self.n) or ids.device != self.device:
                raise ValueError(f"the TokenSort must be of {T} tokens, one choice of {self.n} each, on {self.device}")
            a.d_order, a.d_offsets, a.d_tiles = ids._s.d_order, ids._s.d_offsets, ids._s.d_tiles
            ids = (ids.ids if ids.ids.dim() == 1 else ids.ids[:, 0]).contiguous()
        wide = isinstance(ids, torch.Tensor) and ids.dtype is torch.int64
        a.idx_bytes, a.d_idx = 8 if wide else 4, _vector("ids", ids, T, torch.int64 if wide else torch.int32, self.device)
        if a.d_idx is None and T:
            raise ValueError("ids is missing")
        return ids

    def _ws(self, T, backward):
        return _ws_cached(self._ws_of, (self.in_features, self.out_features, self.rank, self.n, T, backward),
                          L.ecf_adapter_workspace_bytes)

    def forward(self, x, ids, residual=None, out=None, save=False):
        """out [T, out_features] (into `out` if given, which may be the residual); with save,
        (out, h): also h [T, rank] = down[a] x[t] in fp32, for backward()."""
        T = self._matrix_of("x", x)
        a = L.AdapterArgs.from_buffer_copy(self._a)
        a.d_x, a.ld_x = _matrix("x", x, T, self.in_features, self.dtype, self.device)
        ids = self._ids(a, ids, T)
        if residual is not None:
            a.d_residual, a.ld_residual = _matrix("residual", residual, T, self.out_features, self.out_dtype, self.device)
        if (self._learns or x.requires_grad or residual is not None and residual.requires_grad) and not save:
            _warn_untracked("LowRankAdapters")
        y, a.d_out, a.ld_out = self._out("out", out, T, self.out_features, self.out_dtype)
        if save:
            h, a.d_h, _ = self._out("h", None, T, self.rank, torch.float32)
        self._run(L.ecf_adapter_forward, a, T, self._ws(T, 0))
        return (y, h) if save else y

    def backward(self, x, ids, h, dout, residual=None, w_grad_dtype=None, dx=None, need_dx=True, need_dw=True):
        """(dx, ddown, dup) for the gradient dout of out, from the x and ids of the forward call
        and the h it saved.  residual: a gradient that x has already (the projection's), added
        to dx (which it may be); dx is None without need_dx, ddown and dup without need_dw;
        they come in w_grad_dtype (the weights' type, or torch.float32), zeros for an
        adapter of no token.  The forward residual's gradient is dout itself."""
        T = self._matrix_of("x", x)
        a = L.AdapterArgs.from_buffer_copy(self._a)
        gd = self.dtype if w_grad_dtype is None else w_grad_dtype
        if gd is not self.dtype and gd is not torch.float32:
            raise ValueError(f"w_grad_dtype must be {self.dtype} or torch.float32, got {gd}")
        a.wgrad_dtype = _DENSE_DT[gd]
        a.d_x, a.ld_x = _matrix("x", x, T, self.in_features, self.dtype, self.device)
        ids = self._ids(a, ids, T)
        a.d_dout, a.ld_dout = _matrix("dout", dout, T, self.out_features, self.out_dtype, self.device)
        down = up = None
        if need_dx:
            if residual is not None:
                a.d_residual, a.ld_residual = _matrix("residual", residual, T, self.in_features, self.dtype, self.device)
            dx, a.d_dx, a.ld_dx = self._out("dx", dx, T, self.in_features, self.dtype)
        elif dx is not None or residual is not None:
            raise ValueError("dx or residual is given but need_dx is false")
        if need_dw:
            hp, ld = _matrix("h", h, T, self.rank, torch.float32, self.device)
            if ld != self.rank:
                raise ValueError(f"h must be contiguous (row stride {ld})")
            a.d_h = hp
            down, up = self._empty[gd](self.down.shape), self._empty[gd](self.up.shape)
            a.d_da, a.d_db = down.data_ptr(), up.data_ptr()
        self._run(L.ecf_adapter_backward, a, T, self._ws(T, 1))
        return dx, down, up
