"""Operators of the vision tower between the PatchEmbed and the PatchMerger:
rotary positions, layer norm and attention inside each frame, with their
gradients (``pe_vision_positions``, ``pe_rope``, ``pe_layernorm_*`` and
``pe_attention_*`` of the C ABI, include/pe.h).

The functions run on the tensors' own device, on ``stream`` (a torch stream or
a raw handle) or, without one, on that device's current stream.  Outputs and
workspaces are allocated on the stream the call runs on, so calls on several
streams share nothing and a call can be captured into a CUDA graph.  Nothing
here records an autograd graph: the gradient calls are functions of their own.
"""
from __future__ import annotations

import contextlib
from typing import Optional, Sequence, Tuple

import torch

from . import _binding as B
from . import _dt, _need, _raw_stream

__all__ = ["vision_positions", "rope", "layer_norm", "layer_norm_backward", "Attention"]

_HERE = contextlib.nullcontext()


def _on(device: int, stream):
    """(context in which `device` and `stream` are current, raw stream handle)."""
    if stream is None:
        if torch.cuda.current_device() == device:
            return _HERE, _raw(device)
        return torch.cuda.device(device), _raw(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    if stream.device.index != device:
        raise ValueError(f"stream is on cuda:{stream.device.index}, the tensors on cuda:{device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _raw(device: int) -> int:
    if _raw_stream is not None:
        return int(_raw_stream(device))
    return torch.cuda.current_stream(device).cuda_stream


def _device(t: torch.Tensor, name: str) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _dense(t: torch.Tensor, name: str, device: int, shape: Optional[Sequence[int]] = None,
           dtype: Optional[torch.dtype] = None) -> int:
    """Data pointer of a contiguous tensor on `device`."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}; expected cuda:{device}")
    if shape is not None:
        _need(t, shape, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}; expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, device: int, dtype: torch.dtype, shape: Sequence[int]) -> B.pe_heads:
    """A [rows, heads, D] tensor whose last axis is contiguous."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}; expected cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}; expected {dtype}")
    _need(t, shape, name)
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"the last axis of {name} must be contiguous")
    return B.pe_heads(t.data_ptr(), s[0], s[1])


def vision_positions(grid_thw: Sequence[Sequence[int]], merge: int = 2, device=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(pos, cu_seqlens) of the items' patch rows in the forward calls' order:
    pos is int32 [3, N], the (t, h, w) of every row; cu_seqlens is int32
    [frames + 1], the first row of every frame and N.  `device` defaults to the
    current CUDA device."""
    for g in grid_thw:
        if len(g) != 3:
            raise ValueError("every grid_thw entry must be (t, h, w)")
    grids = [int(v) for g in grid_thw for v in g]
    n = sum(grids[i] * grids[i + 1] * grids[i + 2] for i in range(0, len(grids), 3))
    if any(v < 1 for v in grids) or n >= 2 ** 31:
        raise ValueError("grid_thw entries must be positive and their patches fewer than 2^31")
    dev = torch.cuda.current_device() if device is None else torch.device(device).index
    if dev is None:
        dev = torch.cuda.current_device()
    ctx, st = _on(dev, stream)
    with ctx:
        pos = torch.empty((3, n), dtype=torch.int32, device=dev)
        cu = torch.empty(sum(grids[0::3]) + 1, dtype=torch.int32, device=dev)
        B.pe_vision_positions([grids[i:i + 3] for i in range(0, len(grids), 3)], merge, pos.data_ptr(), cu.data_ptr(),
                              st)
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
    dev = _device(q, "q")
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [N, heads, D]")
    n, hq, d = q.shape
    hk = 0 if k is None else k.shape[1]
    if pos.dim() != 2 or pos.shape[0] != len(sections):
        raise ValueError(f"pos must be [{len(sections)}, N]; got {tuple(pos.shape)}")
    pos_ptr = _dense(pos, "pos", dev, (len(sections), n), torch.int32)
    dt = _dt(q.dtype)
    ctx, st = _on(dev, stream)
    with ctx:
        if out_q is None:
            out_q = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
        none = B.pe_heads(None, 0, 0)
        qs, qo = _heads(q, "q", dev, q.dtype, (n, hq, d)), _heads(out_q, "out_q", dev, q.dtype, (n, hq, d))
        ks = ko = none
        if k is not None:
            if out_k is None:
                out_k = torch.empty((n, hk, d), dtype=q.dtype, device=q.device)
            ks, ko = _heads(k, "k", dev, q.dtype, (n, hk, d)), _heads(out_k, "out_k", dev, q.dtype, (n, hk, d))
        B.pe_rope(qs, ks, dt, n, hq, hk, d, pos_ptr, sections, float(theta), axial, inverse, qo, ko, st)
    return out_q, out_k if k is not None else None


def _weights(dev: int, E: int, **weights) -> Tuple[list, int]:
    """Pointers of the optional [E] weights, which share one dtype."""
    ptrs, dts = [], set()
    for name, w in weights.items():
        ptrs.append(None if w is None else _dense(w, name, dev, (E,)))
        if w is not None:
            dts.add(w.dtype)
    if len(dts) > 1:
        raise TypeError("the weights must share one dtype")
    return ptrs, _dt(dts.pop()) if dts else B.PE_F32


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None, stats: bool = False, stream=None):
    """Layer norm over the last axis of a contiguous x [..., E]; gamma and beta
    are [E] or None.  With ``stats`` returns (y, mean, rstd), the fp32
    statistics of every row that `layer_norm_backward` takes.  ``out`` may be x."""
    dev = _device(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., E]")
    E, lead = x.shape[-1], x.shape[:-1]
    xp, dt = _dense(x, "x", dev), _dt(x.dtype)
    (g, b), w_dt = _weights(dev, E, gamma=gamma, beta=beta)
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(x)
        op = _dense(out, "out", dev, x.shape, x.dtype)
        mean = torch.empty(lead, dtype=torch.float32, device=x.device) if stats else None
        rstd = torch.empty_like(mean) if stats else None
        B.pe_layernorm_forward(xp, dt, lead.numel(), E, g, b, w_dt, eps, op, mean.data_ptr() if stats else None,
                               rstd.data_ptr() if stats else None, st)
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, weight_grads: bool = True, out: Optional[torch.Tensor] = None,
                        weight_dtype: Optional[torch.dtype] = None, stream=None):
    """(dx, dgamma, dbeta) of `layer_norm` for the gradient dy of its output; the
    weight's gradients are None with ``weight_grads=False``.  They have gamma's
    dtype (``weight_dtype``, or fp32, without a gamma).  ``out`` may be dy or x."""
    dev = _device(x, "x")
    E, lead = x.shape[-1], x.shape[:-1]
    xp, dt = _dense(x, "x", dev), _dt(x.dtype)
    dp = _dense(dy, "dy", dev, x.shape, x.dtype)
    mp, rp = _dense(mean, "mean", dev, lead, torch.float32), _dense(rstd, "rstd", dev, lead, torch.float32)
    (g,), w_dt = _weights(dev, E, gamma=gamma)
    if weight_dtype is not None:
        if gamma is not None and weight_dtype != gamma.dtype:
            raise TypeError("weight_dtype must be gamma's dtype")
        w_dt = _dt(weight_dtype)
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(x)
        op = _dense(out, "out", dev, x.shape, x.dtype)
        dgamma = dbeta = ws = None
        nbytes = 0
        if weight_grads:
            w_type = torch.float32 if w_dt == B.PE_F32 else torch.bfloat16
            dgamma = torch.empty(E, dtype=w_type, device=x.device)
            dbeta = torch.empty_like(dgamma)
            nbytes = max(B.pe_layernorm_backward_workspace(lead.numel(), E), 0)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        B.pe_layernorm_backward(dp, xp, dt, lead.numel(), E, g, w_dt, mp, rp, op,
                                dgamma.data_ptr() if weight_grads else None,
                                dbeta.data_ptr() if weight_grads else None, ws.data_ptr() if weight_grads else None,
                                nbytes, st)
    return out, dgamma, dbeta


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
        for t, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
            if t.dim() != 1 or t.shape[0] < 1:
                raise ValueError(f"{name} must be [n_seq + 1]; got {tuple(t.shape)}")
        if cu_q.shape != cu_k.shape:
            raise ValueError(f"cu_q {tuple(cu_q.shape)} and cu_k {tuple(cu_k.shape)} hold different sequence counts")
        return (cu_q.shape[0] - 1, _dense(cu_q, "cu_q", self.dev, dtype=torch.int32),
                _dense(cu_k, "cu_k", self.dev, dtype=torch.int32))

    def _shapes(self, q, k):
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q, k and v must be [rows, heads, head_dim]")
        return (q.shape[0], self.heads, self.head_dim), (k.shape[0], self.kv_heads, self.head_dim)

    def _workspace(self, n, nq, nk, backward):
        nbytes = max(B.pe_attention_workspace(self.h, n, nq, nk, backward), 0)
        return (torch.empty(nbytes, dtype=torch.uint8, device=self.dev) if nbytes else None), nbytes

    def forward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, lse: bool = True,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """q [Nq, heads, D], k and v [Nk, kv_heads, D] bf16 (any row and head
        strides that are multiples of 8), cu_q and cu_k int32 [n_seq + 1] on the
        device (cu_k None: cu_q).  Returns (out [Nq, heads, D] bf16, lse [heads,
        Nq] fp32 or None).  Rows of no sequence are not written."""
        cu_k = cu_q if cu_k is None else cu_k
        n, cq, ck = self._cu(cu_q, cu_k)
        sq, sk = self._shapes(q, k)
        d, bf = self.dev, torch.bfloat16
        ctx, st = _on(d, stream)
        with ctx:
            if out is None:
                out = torch.empty(sq, dtype=bf, device=d)
            stat = torch.empty((self.heads, sq[0]), dtype=torch.float32, device=d) if lse else None
            ws, nbytes = self._workspace(n, sq[0], sk[0], False)
            B.pe_attention_forward(self.h, n, cq, sq[0], ck, sk[0], _heads(q, "q", d, bf, sq), _heads(k, "k", d, bf, sk),
                                   _heads(v, "v", d, bf, sk), _heads(out, "out", d, bf, sq),
                                   stat.data_ptr() if lse else None, ws.data_ptr() if nbytes else None, nbytes, st)
        return out, stat

    def backward(self, dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                 lse: torch.Tensor, cu_q: torch.Tensor, cu_k: Optional[torch.Tensor] = None,
                 dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                 dv: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(dq, dk, dv) for the gradient dout of out; out and lse are forward's.
        dq, dk and dv may be given (slices of one packed gradient, for instance)."""
        cu_k = cu_q if cu_k is None else cu_k
        n, cq, ck = self._cu(cu_q, cu_k)
        sq, sk = self._shapes(q, k)
        d, bf = self.dev, torch.bfloat16
        lp = _dense(lse, "lse", d, (self.heads, sq[0]), torch.float32)
        ctx, st = _on(d, stream)
        with ctx:
            dq = torch.empty(sq, dtype=bf, device=d) if dq is None else dq
            dk = torch.empty(sk, dtype=bf, device=d) if dk is None else dk
            dv = torch.empty(sk, dtype=bf, device=d) if dv is None else dv
            ws, nbytes = self._workspace(n, sq[0], sk[0], True)
            B.pe_attention_backward(self.h, n, cq, sq[0], ck, sk[0], _heads(q, "q", d, bf, sq), _heads(k, "k", d, bf, sk),
                                    _heads(v, "v", d, bf, sk), _heads(out, "out", d, bf, sq), lp,
                                    _heads(dout, "dout", d, bf, sq), _heads(dq, "dq", d, bf, sq),
                                    _heads(dk, "dk", d, bf, sk), _heads(dv, "dv", d, bf, sk),
                                    ws.data_ptr() if nbytes else None, nbytes, st)
        return dq, dk, dv

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
