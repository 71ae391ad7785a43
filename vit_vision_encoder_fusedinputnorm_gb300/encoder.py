"""Torch-side calls of the encoder-block operators: layer norm, multi-axis rotary, attention.

What runs behind the front end's embeddings: the tower's norms and packed attention
(sequence boundaries from ``FrontEnd.cu_seqlens``) and the language model's rotary positions of
text, images and video.  PyTorch provides device memory and streams; every operator runs in the
library's CUDA kernels (see ``binding``).

The plain functions return gradients explicitly.  ``LayerNorm``, ``MropeRotation`` and
``PackedAttention`` are the same calls as torch autograd functions (of first order), and ``EncoderBlock`` is a
pre-norm transformer block made of them.

A call runs on the current stream, or on ``stream`` (a torch stream or a cudaStream_t), and what it
allocates belongs to that stream.  A tensor made on another stream has to be ready there, as for
any other call.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

_DTYPES = {torch.bfloat16: B.VITFE_BF16, torch.float16: B.VITFE_F16, torch.float32: B.VITFE_F32}
_float32 = torch.float32
_empty, _empty_like = torch.empty, torch.empty_like
# (a torch built without CUDA has neither, nor a tensor that a call would take)
_get_device, _raw_stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))


# A call of these costs a few microseconds beside kernels that may take as few, so the helpers below
# are kept short, and the wrappers call the library's entry points themselves.

def _dtype(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"bfloat16, float16 or float32 tensors are supported, not {t.dtype}")
    return code


def _current(stream, x: torch.Tensor):
    """Make ``stream`` current on x's GPU, so that outputs and workspaces are that stream's memory."""
    device = _device(x)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)      # a handle does not say whose it is
    elif stream.device_index != device:
        raise ValueError(f"the stream is on GPU {stream.device_index}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _launch(name: str, device: int, *args) -> None:
    """Call an entry point on the current stream of ``device``."""
    entry = getattr(B.load(), name)
    if device == _get_device():
        code = entry(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            code = entry(*args, _raw_stream(device))
    if code:
        raise B.VitfeError(name, code)


def _device(x: torch.Tensor, *others) -> int:
    """The GPU that all of the tensors are on."""
    i = x.get_device()
    if i < 0:
        raise ValueError("CUDA tensors are needed")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError("all tensors have to be on one device")
    return i


def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _words(t: Optional[torch.Tensor], count: int, name: str) -> Optional[int]:
    """Address of `count` int32 that a kernel reads or writes, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() < count or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 [{count}] tensor is needed")
    return t.data_ptr()


def _rows(x: torch.Tensor, name: str) -> int:
    """Row stride of a [rows][width] tensor whose rows are contiguous."""
    if x.dim() != 2:
        raise ValueError(f"{name}: a [rows][width] tensor is needed, not {tuple(x.shape)}")
    row, col = x.stride()
    if col == 1 and row >= x.shape[1]:
        return row
    rows, width = x.shape
    if col != 1 and rows and width > 1:
        raise ValueError(f"{name}: its rows have to be contiguous")
    return row if rows > 1 else width


def _heads(x: torch.Tensor, name: str) -> int:
    """Row stride of a [rows][heads][head_dim] tensor whose rows are contiguous."""
    if x.dim() != 3:
        raise ValueError(f"{name}: a [rows][heads][head_dim] tensor is needed, not {tuple(x.shape)}")
    rows, heads, dim = x.shape
    row, head, col = x.stride()
    if rows and ((col != 1 and dim > 1) or (head != dim and heads > 1)):
        raise ValueError(f"{name}: its rows have to be contiguous")
    return row if rows > 1 else heads * dim


def _like(x: torch.Tensor) -> torch.Tensor:
    return _empty_like(x) if x.is_contiguous() else _empty(x.shape, dtype=x.dtype, device=x.device)


def _target(x: torch.Tensor, out: Optional[torch.Tensor], name: str) -> torch.Tensor:
    if out is None:
        return _like(x)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{name}: the input's shape and type are needed")
    return out


def _vector(v: torch.Tensor, width: int, name: str, dtype: Optional[torch.dtype] = None) -> int:
    """Address of a contiguous [width] tensor."""
    if v.dim() != 1 or v.shape[0] != width or not v.is_contiguous() or (dtype is not None and v.dtype != dtype):
        raise ValueError(f"{name}: a contiguous [{width}] tensor{f' of {dtype}' if dtype else ''} is needed")
    return v.data_ptr()


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, stats: bool = False, stream=None):
    """Layer norm over the rows of x [rows][width]; with ``stats``: (y, mean, rstd) for the backward pass."""
    if stream is not None:
        with _current(stream, x):
            return layer_norm(x, weight, bias, eps, out, stats)
    stride = _rows(x, "x")
    rows, width = x.shape
    device = _device(x, weight, bias, out)
    w = b = None
    kind = B.VITFE_F32
    if weight is not None:
        w, kind = _vector(weight, width, "weight"), _dtype(weight)
    if bias is not None:
        b = _vector(bias, width, "bias", None if weight is None else weight.dtype)
        kind = _dtype(bias)
    if out is None:
        out = _like(x)
        out_stride = width
    else:
        out_stride = _rows(_target(x, out, "out"), "out")
    if not stats:
        _launch("vitfe_layer_norm", device, x.data_ptr(), stride, _dtype(x), rows, width, w, b, kind, eps,
                out.data_ptr(), out_stride, None, None)
        return out
    mean = _empty(rows, dtype=_float32, device=x.device)
    rstd = _empty_like(mean)
    _launch("vitfe_layer_norm", device, x.data_ptr(), stride, _dtype(x), rows, width, w, b, kind, eps, out.data_ptr(),
            out_stride, mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def layer_norm_backward(dout, x, mean, rstd, weight=None, params: bool = True, stream=None):
    """(dx, dweight, dbias) of layer_norm; the last two float32, or None without ``params``."""
    if stream is not None:
        with _current(stream, x):
            return layer_norm_backward(dout, x, mean, rstd, weight, params)
    stride = _rows(x, "x")
    rows, width = x.shape
    device = _device(x, dout, mean, rstd, weight)
    if dout.shape != x.shape or dout.dtype != x.dtype:
        raise ValueError("dout: x's shape and type are needed")
    w, kind = (None, B.VITFE_F32) if weight is None else (_vector(weight, width, "weight"), _dtype(weight))
    m, r = _vector(mean, rows, "mean", _float32), _vector(rstd, rows, "rstd", _float32)
    dx = _like(x)
    if not params:
        _launch("vitfe_layer_norm_backward", device, dout.data_ptr(), _rows(dout, "dout"), x.data_ptr(), stride,
                _dtype(x), rows, width, w, kind, m, r, dx.data_ptr(), width, None, None, None, 0)
        return dx, None, None
    dweight = _empty(width, dtype=_float32, device=x.device)
    dbias = _empty_like(dweight)
    size = B.vitfe_layer_norm_workspace(rows, width)
    work = _empty(size, dtype=torch.uint8, device=x.device)
    _launch("vitfe_layer_norm_backward", device, dout.data_ptr(), _rows(dout, "dout"), x.data_ptr(), stride, _dtype(x),
            rows, width, w, kind, m, r, dx.data_ptr(), width, dweight.data_ptr(), dbias.data_ptr(), work.data_ptr(),
            size)
    return dx, dweight, dbias


# ------------------------------------------------------------------ rotary positions

def section_axes(sections: Sequence[int], interleaved: bool = False) -> list:
    """The axis of each rotated pair, for sections of (time, height, width, ...) pairs.

    In order: the first section's pairs, then the second's, and so on.  Interleaved: axis a > 0
    takes the pairs a, a + n, a + 2n, ... (n axes) until its section is used up, axis 0 the rest.
    """
    n, total = len(sections), sum(sections)
    if not interleaved:
        return [a for a in range(n) for _ in range(sections[a])]
    return [i % n if i % n and i < n * sections[i % n] else 0 for i in range(total)]


def mrope_positions(spans, n_spans, items, n_items, rows: int, merge: int = 2, pos=None, status=None, stream=None):
    """int32 [3][rows] positions of a packed prompt (vitfe_mrope_positions).

    spans: int32 [capacity][4] on the device (first, text, item, step); items: the item table of
    ``FrontEnd.upload`` (24 bytes an item), or None.
    """
    if stream is not None:
        with _current(stream, spans):
            return mrope_positions(spans, n_spans, items, n_items, rows, merge, pos, status)
    device = _device(spans, n_spans, items, n_items, pos, status)
    if spans.dtype != torch.int32 or spans.dim() != 2 or spans.shape[1] != 4 or not spans.is_contiguous():
        raise ValueError("spans: a contiguous int32 [capacity][4] tensor is needed")
    capacity = 0
    if items is not None:
        if not items.is_contiguous():
            raise ValueError("items: a contiguous table is needed")
        capacity = items.numel() * items.element_size() // 24
    if pos is None:
        pos = torch.empty((3, rows), dtype=torch.int32, device=spans.device)
    elif pos.shape != (3, rows) or pos.dtype != torch.int32 or not pos.is_contiguous():
        raise ValueError("pos: a contiguous int32 [3][rows] tensor is needed")
    _launch("vitfe_mrope_positions", device, spans.data_ptr(), _words(n_spans, 1, "n_spans"), spans.shape[0],
            _ptr(items), _words(n_items, 1, "n_items"), capacity, merge, rows, pos.data_ptr(),
            _words(status, 2, "status"))
    return pos


def mrope_apply(q, k, pos, axes: Sequence[int], theta: float = 10000.0, inverse: bool = False, q_out=None, k_out=None,
                stream=None):
    """(q, k) rotated: [rows][heads][head_dim] each, either may be None.

    pos: int32 [n axes][rows]; axes: the axis of each pair (``section_axes``), rotary_dim / 2 of
    them.  q_out, k_out: where to write (q and k themselves for in place), else new tensors.
    """
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    if stream is not None:
        with _current(stream, x):
            return mrope_apply(q, k, pos, axes, theta, inverse, q_out, k_out)
    device = _device(x, q, k, pos, q_out, k_out)
    if q is not None:
        q_out = _target(q, q_out, "q_out")
        tq = (q.data_ptr(), q.shape[1], _heads(q, "q"), q_out.data_ptr(), _heads(q_out, "q_out"))
    else:
        tq = (None, 0, 0, None, 0)
    if k is not None:
        if k.dtype != x.dtype or k.dim() != 3 or k.shape[0] != x.shape[0] or k.shape[2] != x.shape[2]:
            raise ValueError("q and k: the same rows, head_dim and type are needed")
        k_out = _target(k, k_out, "k_out")
        tk = (k.data_ptr(), k.shape[1], _heads(k, "k"), k_out.data_ptr(), _heads(k_out, "k_out"))
    else:
        tk = (None, 0, 0, None, 0)
    rows, _, dim = x.shape
    if pos.dtype != torch.int32 or pos.dim() != 2 or pos.shape[1] != rows or not pos.is_contiguous():
        raise ValueError("pos: a contiguous int32 [axes][rows] tensor is needed")
    _launch("vitfe_mrope_apply", device, pos.data_ptr(), pos.shape[0], bytes(axes), 2 * len(axes), theta, bool(inverse),
            rows, dim, _dtype(x), *tq, *tk)
    return q_out, k_out


# ------------------------------------------------------------------ attention

class AttentionPlan:
    """Sequence boundaries of a batch, made into the attention kernels' work list once for all layers.

    cu_q, cu_k: int32 [sequences + 1] on the device (``FrontEnd.cu_seqlens`` gives them; the tower's
    queries and keys share one).  rows_q, rows_k: rows of q and of k, v, padding included.
    """

    def __init__(self, cu_q, cu_k, rows_q: int, rows_k: int, heads_q: int, heads_kv: int, head_dim: int,
                 causal: bool = False, status=None, stream=None):
        self.device = _device(cu_q, cu_k, status)
        self.version = 0
        if cu_q.dim() != 1 or not len(cu_q):
            raise ValueError("cu_q: an int32 [sequences + 1] tensor is needed")
        shape = (rows_q, rows_k, len(cu_q) - 1, heads_q, heads_kv, head_dim, int(causal))
        # one shape for each type that a call may have: workspaces do not depend on it
        self._shapes = {t: B.AttentionShape(*shape, _DTYPES[t]) for t in (torch.bfloat16, torch.float16)}
        self.shape = self._shapes[torch.bfloat16]
        self._q, self._k = (rows_q, heads_q, head_dim), (rows_k, heads_kv, head_dim)
        self._work = B.vitfe_attention_workspace(self.shape)
        self._work_backward = B.vitfe_attention_backward_workspace(self.shape)
        with _current(stream if stream is not None else torch.cuda.current_stream(cu_q.device), cu_q):
            size = B.vitfe_attention_plan_bytes(self.shape)
            self.buffer = torch.empty(max(size, 16), dtype=torch.uint8, device=cu_q.device)
            self._home = torch.cuda.current_stream(cu_q.device).cuda_stream
            self.update(cu_q, cu_k, status)

    def update(self, cu_q, cu_k, status=None, stream=None) -> None:
        """Plan new boundaries in the same buffer (the shape stays: a captured graph replays this).

        What was attended under the boundaries before keeps no copy of them: ``PackedAttention`` refuses
        gradients across an update (``version`` counts them; a graph's replays are not seen).
        """
        if stream is not None:
            with _current(stream, cu_q):
                return self.update(cu_q, cu_k, status)
        device = _device(self.buffer, cu_q, cu_k, status)
        for c in (cu_q, cu_k):
            if c.dtype != torch.int32 or not c.is_contiguous() or c.shape != (self.shape.max_seqs + 1,):
                raise ValueError(f"cu_q, cu_k: contiguous int32 [{self.shape.max_seqs + 1}] tensors are needed")
        status = _words(status, 2, "status")
        self.version += 1
        _launch("vitfe_attention_plan", device, self.shape, cu_q.data_ptr(), cu_k.data_ptr(), self.buffer.data_ptr(),
                status)

    def address(self, device: int) -> int:
        """The buffer's address for a call on the current stream; a plan that goes away before that call
        has run leaves its memory to it, whichever stream it was made on."""
        if _raw_stream(device) != self._home:
            self.buffer.record_stream(torch.cuda.current_stream(device))
        return self.buffer.data_ptr()

    def of(self, q, k, v) -> "B.AttentionShape":
        """The shape of a call with these tensors; raises where they do not fit the plan."""
        if q.shape != self._q:
            raise ValueError(f"q: {self._q} is planned, not {tuple(q.shape)}")
        if k.shape != self._k or v.shape != self._k:
            raise ValueError(f"k, v: {self._k} is planned, not {tuple(k.shape)}, {tuple(v.shape)}")
        dtype = q.dtype
        if k.dtype != dtype or v.dtype != dtype or dtype not in self._shapes:
            raise ValueError("q, k, v: one type, bfloat16 or float16, is needed")
        return self._shapes[dtype]


def attention(q, k, v, plan: AttentionPlan, scale: Optional[float] = None, lse: bool = False, out=None, status=None,
              stream=None):
    """softmax(scale q k^T) v over the plan's sequences; with ``lse``: (out, lse float32 [rows][heads])."""
    if stream is not None:
        with _current(stream, q):
            return attention(q, k, v, plan, scale, lse, out, status)
    shape = plan.of(q, k, v)
    device = _device(plan.buffer, q, k, v, out, status)
    out = _target(q, out, "out")
    sums = _empty(plan._q[:2], dtype=_float32, device=q.device) if lse else None
    work = _empty(plan._work, dtype=torch.uint8, device=q.device) if plan._work else None
    _launch("vitfe_attention", device, shape, plan.address(device), q.data_ptr(), _heads(q, "q"), k.data_ptr(),
            _heads(k, "k"), v.data_ptr(), _heads(v, "v"), q.shape[2] ** -0.5 if scale is None else scale,
            out.data_ptr(), _heads(out, "out"), _ptr(sums), _ptr(work), _words(status, 2, "status"))
    return (out, sums) if lse else out


def attention_backward(dout, q, k, v, out, lse, plan: AttentionPlan, scale: Optional[float] = None, status=None,
                       stream=None):
    """(dq, dk, dv) of attention; ``out`` and ``lse`` are the forward pass's."""
    if stream is not None:
        with _current(stream, q):
            return attention_backward(dout, q, k, v, out, lse, plan, scale, status)
    shape = plan.of(q, k, v)
    device = _device(plan.buffer, dout, q, k, v, out, lse, status)
    for t, name in ((dout, "dout"), (out, "out")):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name}: q's shape and type are needed")
    if lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse: the forward pass's float32 [rows][heads] is needed")
    dq, dk, dv = _like(q), _like(k), _like(v)
    work = _empty(plan._work_backward, dtype=torch.uint8, device=q.device) if plan._work_backward else None
    _launch("vitfe_attention_backward", device, shape, plan.address(device), dout.data_ptr(), _heads(dout, "dout"),
            q.data_ptr(), _heads(q, "q"), k.data_ptr(), _heads(k, "k"), v.data_ptr(), _heads(v, "v"), out.data_ptr(),
            _heads(out, "out"), lse.data_ptr(), q.shape[2] ** -0.5 if scale is None else scale, dq.data_ptr(),
            _heads(dq, "dq"), dk.data_ptr(), _heads(dk, "dk"), dv.data_ptr(), _heads(dv, "dv"), _ptr(work),
            _words(status, 2, "status"))
    return dq, dk, dv


# ------------------------------------------------------------------ autograd

class LayerNorm(torch.autograd.Function):
    """``LayerNorm.apply(x, weight, bias, eps)``: layer_norm with its gradients."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm(x, weight, bias, eps, stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        params = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dw, db = layer_norm_backward(dy.contiguous(), x, mean, rstd, weight, params=params)
        return (dx, dw.to(weight.dtype) if ctx.needs_input_grad[1] else None,
                db.to(ctx.bias_dtype) if ctx.needs_input_grad[2] else None, None)


class MropeRotation(torch.autograd.Function):
    """``MropeRotation.apply(q, k, pos, axes, theta)``: mrope_apply; its gradient is the inverse rotation.

    q or k may be None, as there.
    """

    @staticmethod
    def forward(ctx, q, k, pos, axes, theta):
        ctx.save_for_backward(pos)
        ctx.axes, ctx.theta = axes, theta
        return mrope_apply(q, k, pos, axes, theta)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        dq, dk = (None if g is None else g.contiguous() for g in (dq, dk))
        dq, dk = mrope_apply(dq, dk, ctx.saved_tensors[0], ctx.axes, ctx.theta, inverse=True)
        return dq, dk, None, None, None


class TableRotation(torch.autograd.Function):
    """``TableRotation.apply(x, cos, sin)``: vitfe_rope_apply with the tower's tables, out of place.

    x: bfloat16 [rows][heads][head_dim]; cos, sin: float32 [rows][head_dim / 2].
    """

    @staticmethod
    def _turn(x, cos, sin):
        if x.dtype != torch.bfloat16:
            raise TypeError(f"x: a bfloat16 tensor is needed, not {x.dtype}")
        if x.dim() != 3:
            raise ValueError(f"x: a [rows][heads][head_dim] tensor is needed, not {tuple(x.shape)}")
        for t, name in ((cos, "cos"), (sin, "sin")):
            if (t.dtype != _float32 or t.dim() != 2 or t.shape[0] < x.shape[0] or 2 * t.shape[1] != x.shape[2]
                    or not t.is_contiguous()):
                raise ValueError(f"{name}: a contiguous float32 {[x.shape[0], x.shape[2] // 2]} tensor is needed")
        _device(x, cos, sin)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device).copy_(x)
        with torch.cuda.device(x.device):
            B.vitfe_rope_apply(cos, sin, x.shape[0], x.shape[2], y, x.shape[1], _heads(y, "x"), None, 0, 0,
                               torch.cuda.current_stream(x.device))
        return y

    @staticmethod
    def forward(ctx, x, cos, sin):
        ctx.save_for_backward(cos, sin)
        return TableRotation._turn(x, cos, sin)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        cos, sin = ctx.saved_tensors
        return TableRotation._turn(dy, cos, -sin), None, None


class PackedAttention(torch.autograd.Function):
    """``PackedAttention.apply(q, k, v, plan, scale)``: attention with its gradients."""

    @staticmethod
    def forward(ctx, q, k, v, plan, scale):
        out, lse = attention(q, k, v, plan, scale, lse=True)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.plan, ctx.scale, ctx.version = plan, scale, plan.version
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        if ctx.plan.version != ctx.version:
            raise RuntimeError("the plan was updated since the forward pass: its gradients need the boundaries of then")
        dq, dk, dv = attention_backward(dout.contiguous(), q, k, v, out, lse, ctx.plan, ctx.scale)
        return dq, dk, dv, None, None


class EncoderBlock(torch.nn.Module):
    """A pre-norm transformer block of the vision tower, on packed rows.

    x + proj(attention(rotate(q), rotate(k), v)), then x + mlp: the rows are the front end's
    embeddings, cos and sin its RoPE tables, and the plan is made of its ``cu_seqlens``.  The
    projections are torch's matrix products; norms, rotation and attention are the library's.
    In bfloat16, as the tower's rotation is.
    """

    def __init__(self, hidden: int, heads: int, mlp: int, eps: float = 1e-6, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        if dtype != torch.bfloat16:
            raise TypeError(f"the block is in bfloat16, not {dtype}")
        if hidden % heads or (hidden // heads) % 8:
            raise ValueError("hidden has to be heads times a multiple of 8")
        self.heads, self.eps = heads, eps
        kw = {"dtype": dtype, "device": device}
        self.norm1_weight = torch.nn.Parameter(torch.ones(hidden, **kw))
        self.norm1_bias = torch.nn.Parameter(torch.zeros(hidden, **kw))
        self.norm2_weight = torch.nn.Parameter(torch.ones(hidden, **kw))
        self.norm2_bias = torch.nn.Parameter(torch.zeros(hidden, **kw))
        self.qkv = torch.nn.Linear(hidden, 3 * hidden, **kw)
        self.proj = torch.nn.Linear(hidden, hidden, **kw)
        self.fc1 = torch.nn.Linear(hidden, mlp, **kw)
        self.fc2 = torch.nn.Linear(mlp, hidden, **kw)

    def forward(self, x, cos, sin, plan: AttentionPlan):
        rows, hidden = x.shape
        h = LayerNorm.apply(x, self.norm1_weight, self.norm1_bias, self.eps)
        q, k, v = self.qkv(h).view(rows, 3 * self.heads, hidden // self.heads).split(self.heads, dim=1)
        q, k = TableRotation.apply(q, cos, sin), TableRotation.apply(k, cos, sin)
        a = PackedAttention.apply(q, k, v, plan, None)
        x = x + self.proj(a.reshape(rows, hidden))
        h = LayerNorm.apply(x, self.norm2_weight, self.norm2_bias, self.eps)
        return x + self.fc2(torch.nn.functional.gelu(self.fc1(h), approximate="tanh"))
