"""Operators of the vision tower between the PatchEmbed and the PatchMerger:
rotary positions, layer norm and attention inside each frame, with their
gradients (``pe_vision_positions``, ``pe_rope``, ``pe_layernorm_*`` and
``pe_attention_*`` of the C ABI, include/pe.h).

The functions run on the tensors' own device, on ``stream`` (a torch stream or
a raw handle) or, without one, on that device's current stream.  Outputs and
workspaces are allocated on the stream the call runs on, so calls on several
streams share nothing and a call can be captured into a CUDA graph.

`rope`, `layer_norm` and `Attention.forward` are differentiable: with grad mode
on and an input that requires grad they are recorded, and torch's backward pass
makes the gradient calls below, which can also be made by hand (they are not
recorded themselves).  A call that is recorded takes no output tensor.  Writes
to output tensors count as in-place changes for autograd's checks.  As with
torch's own operators, a backward pass can be captured while no eager graph of
its leaves lives.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _binding as B
from . import _dt, _need, _raw_stream

__all__ = ["vision_positions", "rope", "layer_norm", "layer_norm_backward", "Attention"]

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_NONE = B.pe_heads(None, 0, 0)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_grad_on = torch.is_grad_enabled


def _no_outputs(*outs: Optional[torch.Tensor]) -> None:
    if any(t is not None for t in outs):
        raise ValueError("a call that autograd records takes no output tensors: an input (or output) requires grad; "
                         "leave them out, or call under torch.no_grad()")


def _elsewhere(device: int, stream) -> bool:
    """Whether a call has to enter another device or stream first (`_on`)."""
    return stream is not None or (device >= 0 and device != _current_device())


def _on(device: int, stream):
    """Context in which `device` and `stream` (None: the device's current one) are current."""
    if device < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    if stream.device.index != device:
        raise ValueError(f"stream is on cuda:{stream.device.index}, the tensors on cuda:{device}")
    return torch.cuda.stream(stream)


def _raw(device: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _dense(t: torch.Tensor, name: str, device: int, shape=None, dtype: Optional[torch.dtype] = None) -> int:
    """Data pointer of a contiguous tensor on `device`."""
    if (t.get_device() == device >= 0 and (shape is None or t.shape == shape)
            and (dtype is None or t.dtype == dtype) and t.is_contiguous()):
        return t.data_ptr()
    _place(t, name, device)
    if shape is not None:
        _need(t, shape, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}; expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _place(t: torch.Tensor, name: str, device: int) -> None:
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}; expected cuda:{device}")


def _heads(t: torch.Tensor, name: str, device: int, dtype: torch.dtype, shape) -> B.pe_heads:
    """A [rows, heads, D] tensor whose last axis is contiguous."""
    if not (t.get_device() == device >= 0 and t.dtype == dtype and t.shape == shape):
        _place(t, name, device)
        if t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}; expected {dtype}")
        _need(t, shape, name)
    row, head, one = t.stride()
    if one != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"the last axis of {name} must be contiguous")
    return B.pe_heads(t.data_ptr(), row, head)


def vision_positions(grid_thw: Sequence[Sequence[int]], merge: int = 2, device=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(pos, cu_seqlens) of the items' patch rows in the forward calls' order:
    pos is int32 [3, N], the (t, h, w) of every row; cu_seqlens is int32
    [frames + 1], the first row of every frame and N.  `device` defaults to the
    current CUDA device."""
    grids, n, frames = [], 0, 0
    for g in grid_thw:
        if len(g) != 3:
            raise ValueError("every grid_thw entry must be (t, h, w)")
        t, h, w = int(g[0]), int(g[1]), int(g[2])
        if t < 1 or h < 1 or w < 1:
            raise ValueError("grid_thw entries must be positive")
        grids += (t, h, w)
        n += t * h * w
        frames += t
    if n >= 2 ** 31:
        raise ValueError("the grids hold 2^31 patches or more")
    dev = None
    if device is not None:
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"device must be a CUDA device; got {device}")
        dev = device.index
    if dev is None:
        dev = _current_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return vision_positions(grid_thw, merge, dev)
    where = torch.device("cuda", dev)
    pos = torch.empty(3, n, dtype=_I32, device=where)
    cu = pos.new_empty(frames + 1)
    B.pe_vision_positions(grids, merge, pos.data_ptr(), cu.data_ptr(), _raw(dev))
    return pos, cu


def rope(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, sections: Sequence[int], theta: float = 10000.0,
         axial: bool = False, inverse: bool = False, out_q: Optional[torch.Tensor] = None,
         out_k: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions on q [N, Hq, D] and k [N, Hk, D] (or None) in one launch.

    pos is int32 [axes, N]; sections[a] pairs of each head turn by the positions
    of axis a.  Pair i holds elements i and i + sum(sections); its rate is
    theta^(-i/sum(sections)), or with ``axial`` theta^(-j/sections[a]) for the
    j-th pair of axis a.  The vision tower uses axial with sections
    (D/4, D/4) on pos[1:] of `vision_positions`; M-RoPE sections (16, 24, 24).
    ``inverse`` turns back, which is the gradient.  Pass ``out_q=q`` (and
    ``out_k=k``) to work in place."""
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rope(q, k, pos, sections, theta, axial, inverse, out_q, out_k)
    if _grad_on() and (q.requires_grad or (k is not None and k.requires_grad)
                       or (out_q is not None and out_q.requires_grad) or (out_k is not None and out_k.requires_grad)):
        _no_outputs(out_q, out_k)
        return _Rope.apply(q, k, pos, tuple(sections), theta, axial, inverse)
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [N, heads, D]")
    if pos.dim() != 2 or pos.shape[0] != len(sections):
        raise ValueError(f"pos must be [{len(sections)}, N]; got {tuple(pos.shape)}")
    dtype, shape = q.dtype, q.shape
    n, hq, d = shape
    dt = _dt(dtype)
    pos_ptr = _dense(pos, "pos", dev, (len(sections), n), _I32)
    qs = _heads(q, "q", dev, dtype, shape)
    if out_q is None:
        out_q = q.new_empty(shape)
        qo = B.pe_heads(out_q.data_ptr(), hq * d, d)
    else:
        qo = _heads(out_q, "out_q", dev, dtype, shape)
        increment_version(out_q)
    hk, ks, ko = 0, _NONE, _NONE
    if k is not None:
        hk = k.shape[1]
        k_shape = (n, hk, d)
        ks = _heads(k, "k", dev, dtype, k_shape)
        if out_k is None:
            out_k = k.new_empty(k_shape)
            ko = B.pe_heads(out_k.data_ptr(), hk * d, d)
        else:
            ko = _heads(out_k, "out_k", dev, dtype, k_shape)
            increment_version(out_k)
    B.pe_rope(qs, ks, dt, n, hq, hk, d, pos_ptr, sections, theta, axial, inverse, qo, ko, _raw(dev))
    return out_q, out_k if k is not None else None


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, pos, sections, theta, axial, inverse):
        ctx.save_for_backward(pos)
        ctx.how, ctx.with_k = (sections, theta, axial, not inverse), k is not None
        return rope(q, k, pos, sections, theta, axial, inverse)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        pos, = ctx.saved_tensors
        dq, dk = (g if g is None or g.stride(-1) == 1 else g.contiguous() for g in (dq, dk))
        dq, dk = rope(dq, dk if ctx.with_k else None, pos, *ctx.how)
        return dq, dk, None, None, None, None, None


def _weights(dev: int, E: int, gamma, beta=None) -> Tuple[Optional[int], Optional[int], int]:
    """Pointers of the optional [E] weights, and their dtype."""
    if gamma is not None and beta is not None and beta.dtype != gamma.dtype:
        raise TypeError("the weights must share one dtype")
    g = None if gamma is None else _dense(gamma, "gamma", dev, (E,))
    b = None if beta is None else _dense(beta, "beta", dev, (E,))
    if gamma is not None:
        return g, b, _dt(gamma.dtype)
    return g, b, B.PE_F32 if beta is None else _dt(beta.dtype)


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None, stats: bool = False, stream=None):
    """Layer norm over the last axis of a contiguous x [..., E]; gamma and beta
    are [E] or None.  With ``stats`` returns (y, mean, rstd), the fp32
    statistics of every row that `layer_norm_backward` takes.  ``out`` may be x."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm(x, gamma, beta, eps, out, stats)
    if _grad_on() and (x.requires_grad or (gamma is not None and gamma.requires_grad)
                       or (beta is not None and beta.requires_grad) or (out is not None and out.requires_grad)):
        _no_outputs(out)
        y, mean, rstd = _LayerNorm.apply(x, gamma, beta, eps)
        return (y, mean, rstd) if stats else y
    if x.dim() < 1:
        raise ValueError("x must be [..., E]")
    shape = x.shape
    E, lead = shape[-1], shape[:-1]
    dtype = x.dtype
    xp, dt = _dense(x, "x", dev), _dt(dtype)
    g, b, w_dt = _weights(dev, E, gamma, beta)
    if out is None:
        out = x.new_empty(shape)
        op = out.data_ptr()
    else:
        op = _dense(out, "out", dev, shape, dtype)
        increment_version(out)
    mean = rstd = mp = rp = None
    if stats:
        mean, rstd = x.new_empty(lead, dtype=_F32), x.new_empty(lead, dtype=_F32)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    B.pe_layernorm_forward(xp, dt, lead.numel(), E, g, b, w_dt, eps, op, mp, rp, _raw(dev))
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, weight_grads: bool = True, out: Optional[torch.Tensor] = None,
                        weight_dtype: Optional[torch.dtype] = None, stream=None):
    """(dx, dgamma, dbeta) of `layer_norm` for the gradient dy of its output; the
    weight's gradients are None with ``weight_grads=False``.  They have gamma's
    dtype (``weight_dtype``, or fp32, without a gamma).  ``out`` may be dy or x."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm_backward(dy, x, gamma, mean, rstd, weight_grads, out, weight_dtype)
    if x.dim() < 1:
        raise ValueError("x must be [..., E]")
    shape = x.shape
    E, lead = shape[-1], shape[:-1]
    n = lead.numel()
    xp, dt = _dense(x, "x", dev), _dt(x.dtype)
    dp = _dense(dy, "dy", dev, shape, x.dtype)
    mp, rp = _dense(mean, "mean", dev, lead, _F32), _dense(rstd, "rstd", dev, lead, _F32)
    g, _, w_dt = _weights(dev, E, gamma)
    if weight_dtype is not None:
        if gamma is not None and weight_dtype != gamma.dtype:
            raise TypeError("weight_dtype must be gamma's dtype")
        w_dt = _dt(weight_dtype)
    if out is None:
        out = x.new_empty(shape)
        op = out.data_ptr()
    else:
        op = _dense(out, "out", dev, shape, x.dtype)
        increment_version(out)
    dgamma = dbeta = gp = bp = ws = None
    nbytes = 0
    if weight_grads:
        dgamma = x.new_empty(E, dtype=_F32 if w_dt == B.PE_F32 else _BF16)
        dbeta = dgamma.new_empty(E)
        nbytes = B.pe_layernorm_backward_workspace(n, E)
        scratch = x.new_empty(max(nbytes, 0), dtype=torch.uint8)
        gp, bp, ws = dgamma.data_ptr(), dbeta.data_ptr(), scratch.data_ptr()
    B.pe_layernorm_backward(dp, xp, dt, n, E, g, w_dt, mp, rp, op, gp, bp, ws, max(nbytes, 0), _raw(dev))
    return out, dgamma, dbeta


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        y, mean, rstd = layer_norm(x, gamma, beta, eps, stats=True)
        ctx.mark_non_differentiable(mean, rstd)
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.weight_dtype = None if beta is None else beta.dtype
        return y, mean, rstd

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dmean, drstd):
        x, gamma, mean, rstd = ctx.saved_tensors
        need_x, need_gamma, need_beta, _ = ctx.needs_input_grad
        dx, dgamma, dbeta = layer_norm_backward(dy.contiguous(), x, gamma, mean, rstd, need_gamma or need_beta,
                                                weight_dtype=ctx.weight_dtype)
        return dx if need_x else None, dgamma if need_gamma else None, dbeta if need_beta else None, None


class Attention:
    """Attention over packed sequences, bf16: each row sees the keys of its own
    sequence (``causal``: up to its own place, sequences aligned at their ends).

    heads query heads share kv_heads key/value heads (default: as many); scale
    defaults to head_dim ** -0.5.  One object may serve calls on several
    streams at once: it holds only the device error word (`last_error`)."""

    def __init__(self, heads: int, kv_heads: Optional[int] = None, head_dim: int = 80, scale: Optional[float] = None,
                 causal: bool = False):
        self.heads, self.kv_heads, self.head_dim = heads, heads if kv_heads is None else kv_heads, head_dim
        self.scale = head_dim ** -0.5 if scale is None else float(scale)
        self.causal = bool(causal)
        self.h = B.pe_attention_create(self.heads, self.kv_heads, head_dim, self.scale, self.causal)
        self.dev = torch.cuda.current_device()   # the device pe_attention_create bound the handle to

    def _cu(self, cu_q, cu_k):
        n = cu_q.shape
        if len(n) != 1 or n[0] < 1:
            raise ValueError(f"cu_q must be [n_seq + 1]; got {tuple(n)}")
        if cu_k is None or cu_k is cu_q:
            cq = _dense(cu_q, "cu_q", self.dev, None, _I32)
            return n[0] - 1, cq, cq
        if cu_k.shape != n:
            raise ValueError(f"cu_q {tuple(n)} and cu_k {tuple(cu_k.shape)} hold different sequence counts")
        return n[0] - 1, _dense(cu_q, "cu_q", self.dev, None, _I32), _dense(cu_k, "cu_k", self.dev, None, _I32)

    def _shapes(self, q, k):
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q, k and v must be [rows, heads, head_dim]")
        return (q.shape[0], self.heads, self.head_dim), (k.shape[0], self.kv_heads, self.head_dim)

    @staticmethod
    def _fresh(t, shape):
        """A tensor this module has just allocated: dense, nothing to check."""
        return B.pe_heads(t.data_ptr(), shape[1] * shape[2], shape[2])

    def _workspace(self, q, n, nq, nk, backward):
        """(tensor or None, pointer or None, bytes)"""
        nbytes = B.pe_attention_workspace(self.h, n, nq, nk, backward)
        if nbytes <= 0:
            return None, None, 0
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        return ws, ws.data_ptr(), nbytes

    def forward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, lse: bool = True,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """q [Nq, heads, D], k and v [Nk, kv_heads, D] bf16 (any row and head
        strides that are multiples of 8), cu_q and cu_k int32 [n_seq + 1] on the
        device (cu_k None: cu_q).  Returns (out [Nq, heads, D] bf16, lse [heads,
        Nq] fp32 or None).  ``out`` must not overlap q, k or v.

        Rows of no sequence (padding before cu_q[0] and behind cu_q[-1]) are not
        written: in a new ``out`` they hold whatever the memory held, NaN perhaps.
        Where a later product reads them, give an ``out`` that holds zeros there.
        (A recorded call and its gradients hold zeros.)"""
        d = self.dev
        n, cq, ck = self._cu(cu_q, cu_k)
        if _elsewhere(d, stream):
            with _on(d, stream):
                return self.forward(q, k, v, cu_q, cu_k, out, lse)
        if _grad_on() and (q.requires_grad or k.requires_grad or v.requires_grad or (out is not None and out.requires_grad)):
            _no_outputs(out)
            out, stat = _Attend.apply(self, q, k, v, cu_q, cu_k)
            return out, stat if lse else None
        sq, sk = self._shapes(q, k)
        qs, ks, vs = _heads(q, "q", d, _BF16, sq), _heads(k, "k", d, _BF16, sk), _heads(v, "v", d, _BF16, sk)
        if out is None:
            out = q.new_empty(sq)
            os = self._fresh(out, sq)
        else:
            os = _heads(out, "out", d, _BF16, sq)
            increment_version(out)
        stat = q.new_empty((self.heads, sq[0]), dtype=_F32) if lse else None
        ws, wp, nbytes = self._workspace(q, n, sq[0], sk[0], False)
        B.pe_attention_forward(self.h, n, cq, sq[0], ck, sk[0], qs, ks, vs, os,
                               stat.data_ptr() if lse else None, wp, nbytes, _raw(d))
        return out, stat

    def backward(self, dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                 lse: torch.Tensor, cu_q: torch.Tensor, cu_k: Optional[torch.Tensor] = None,
                 dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                 dv: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(dq, dk, dv) for the gradient dout of out; out and lse are forward's.
        dq, dk and dv may be given (slices of one packed gradient, for instance);
        none may overlap another tensor of the call.

        Rows of no sequence are not written, as in `forward`: a product over the
        rows of a new gradient (a weight's, for instance) would add what the memory
        held there.  For padded batches give gradients that hold zeros there."""
        d = self.dev
        n, cq, ck = self._cu(cu_q, cu_k)
        if _elsewhere(d, stream):
            with _on(d, stream):
                return self.backward(dout, q, k, v, out, lse, cu_q, cu_k, dq, dk, dv)
        sq, sk = self._shapes(q, k)
        lp = _dense(lse, "lse", d, (self.heads, sq[0]), _F32)
        args = [_heads(t, name, d, _BF16, s) for t, name, s in
                ((q, "q", sq), (k, "k", sk), (v, "v", sk), (out, "out", sq), (dout, "dout", sq))]
        grads = []
        for t, name, s in ((dq, "dq", sq), (dk, "dk", sk), (dv, "dv", sk)):
            if t is None:
                t = q.new_empty(s)
                grads.append((t, self._fresh(t, s)))
            else:
                grads.append((t, _heads(t, name, d, _BF16, s)))
                increment_version(t)
        ws, wp, nbytes = self._workspace(q, n, sq[0], sk[0], True)
        B.pe_attention_backward(self.h, n, cq, sq[0], ck, sk[0], args[0], args[1], args[2], args[3], lp, args[4],
                                grads[0][1], grads[1][1], grads[2][1], wp, nbytes, _raw(d))
        return grads[0][0], grads[1][0], grads[2][0]

    def last_error(self) -> int:
        return B.pe_attention_last_error(self.h)

    def close(self) -> None:
        if getattr(self, "h", None):
            B.pe_attention_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, attention, q, k, v, cu_q, cu_k):
        # rows of no sequence: zeros, here and in the gradients, as what is before and behind reads every row
        out, lse = attention.forward(q, k, v, cu_q, cu_k, q.new_zeros(q.shape))
        ctx.mark_non_differentiable(lse)
        ctx.save_for_backward(q, k, v, out, lse, cu_q, cu_k)
        ctx.attention = attention
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dlse):
        q, k, v, out, lse, cu_q, cu_k = ctx.saved_tensors
        grads = (t.new_zeros(t.shape) for t in (q, k, v))
        return (None, *ctx.attention.backward(dout.contiguous(), q, k, v, out, lse, cu_q, cu_k, *grads), None, None)
