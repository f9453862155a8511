"""Torch-side conveniences over the C ABI: device memory, streams and argument
structs.  Nothing here computes any part of the layer; every step of the
forward pass runs in libecf's kernels (or its host expert threads)."""
from __future__ import annotations

import warnings

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


def _warn_untracked(what):
    """A forward call that something requires gradients of; it gives none where they are on."""
    if torch.is_grad_enabled():
        warnings.warn(f"{what}.forward is outside autograd: its output has no gradient function although the weights or "
                      "an input require gradients.  Run it under torch.no_grad(), and call backward() with the "
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
