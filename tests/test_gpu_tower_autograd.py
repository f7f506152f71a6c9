"""Rotary positions, layer norm and attention under torch's autograd: the gradients
are those of the explicit gradient calls, bit for bit, whatever the layout of the
incoming gradient; output tensors are refused where a call is recorded, and writes
to them elsewhere are seen by autograd's in-place checks."""
from __future__ import annotations

import pytest
import torch

import vlm_vision_patch_b200 as vp
from tests.test_gpu_tower import BF, DEV, F32, _attention_error_words, cu, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_k,dtype", [(True, BF), (False, F32)])
def test_rope_is_recorded(with_k, dtype):
    N, H, D, sec = 133, 3, 80, (20, 20)
    pos = torch.randint(0, 99, (2, N), generator=torch.Generator().manual_seed(1)).int().to(DEV)
    qkv = normal(2, N, 3, H, D, dtype=dtype).requires_grad_()
    q, k = qkv[:, 0], qkv[:, 1] if with_k else None
    a, b = vp.rope(q, k, pos, sec, axial=True)
    plain = vp.rope(q.detach(), k.detach() if with_k else None, pos, sec, axial=True)
    assert torch.equal(a, plain[0]) and (b is None if not with_k else torch.equal(b, plain[1]))
    ga, gb = normal(3, N, H, D, dtype=dtype), normal(4, N, H, D, dtype=dtype)
    ((a * ga).sum() + ((b * gb).sum() if with_k else 0)).backward()
    want = vp.rope(ga, gb, pos, sec, axial=True, inverse=True)
    assert torch.equal(qkv.grad[:, 0], want[0]) and not qkv.grad[:, 2].any()
    assert torch.equal(qkv.grad[:, 1], want[1]) if with_k else not qkv.grad[:, 1].any()
    qkv.grad = None
    vp.rope(qkv[:, 0], None, pos, sec, axial=True)[0].sum().backward()      # a gradient with strides of 0
    assert torch.equal(qkv.grad[:, 0], vp.rope(torch.ones_like(ga), None, pos, sec, axial=True, inverse=True)[0])


@pytest.mark.parametrize("gamma,beta", [(BF, BF), (F32, F32), (None, BF), (F32, None), (None, None)])
def test_layer_norm_is_recorded(gamma, beta):
    N, E = 70, 320
    x = normal(5, N, E, dtype=BF).requires_grad_()
    g = None if gamma is None else normal(6, E, dtype=gamma, mean=1.0).requires_grad_()
    b = None if beta is None else normal(7, E, dtype=beta).requires_grad_()
    y, mean, rstd = vp.layer_norm(x, g, b, 1e-5, stats=True)
    assert y.requires_grad and not mean.requires_grad and not rstd.requires_grad
    dy = normal(8, N, E, dtype=BF)
    y.backward(dy.t().contiguous().t())                                     # columns first
    with torch.no_grad():
        py, pm, pr = vp.layer_norm(x, g, b, 1e-5, stats=True)
        dx, dg, db = vp.layer_norm_backward(dy, x, g, pm, pr, weight_dtype=None if g is not None else beta)
    assert torch.equal(y, py) and not py.requires_grad and torch.equal(x.grad, dx)
    assert g is None or torch.equal(g.grad, dg)
    assert b is None or torch.equal(b.grad, db)
    if g is not None:                                                       # a frozen input: the weights' gradients alone
        g2 = g.detach().clone().requires_grad_()
        vp.layer_norm(x.detach(), g2, None, 1e-5).backward(dy)
        assert torch.equal(g2.grad, dg)


@pytest.mark.parametrize("causal,own_keys", [(False, False), (True, True)])
def test_attention_is_recorded(causal, own_keys):
    D, H, ql = 72, 2, (130, 61)
    kl = (200, 61) if own_keys else ql
    q, k, v = (normal(9 + i, sum(n), H, D, dtype=BF).requires_grad_() for i, n in enumerate((ql, kl, kl)))
    do = normal(12, sum(ql), H, D, dtype=BF)
    att = vp.Attention(H, H, D, causal=causal)
    c, ck = cu(ql), cu(kl) if own_keys else None
    out, none = att.forward(q, k, v, c, ck, lse=False)
    assert none is None
    out.backward(do)
    with torch.no_grad():
        po, lse = att.forward(q, k, v, c, ck)
        want = att.backward(do, q, k, v, po, lse, c, ck)
    assert torch.equal(out, po) and all(torch.equal(t.grad, w) for t, w in zip((q, k, v), want))
    out, lse = att.forward(q.detach(), k.detach(), v, c, ck)                # v alone
    assert not lse.requires_grad
    v.grad = None
    out.sum().backward()
    with torch.no_grad():
        want = att.backward(torch.ones_like(do), q, k, v, po, lse, c, ck)
    assert torch.equal(v.grad, want[2])
    with pytest.raises(RuntimeError):                                       # not differentiable twice
        out, _ = att.forward(q, k, v, c, ck)
        g, = torch.autograd.grad(out.sum(), q, create_graph=True)
        g.sum().backward()


def test_padded_batches_are_recorded_with_zeros():
    """Rows of no sequence hold 0 in the output and in every gradient."""
    D, H, pre, ql, post = 64, 2, 3, (40, 17), 90
    n, mid = pre + sum(ql) + post, slice(pre, pre + sum(ql))
    att = vp.Attention(H, H, D)
    for _ in range(2):
        torch.full((1 << 24,), float("nan"), device=DEV)                    # what new tensors may find
        x = [normal(60 + i, n, H, D, dtype=BF).requires_grad_() for i in range(3)]
        out, _ = att.forward(*x, cu(ql) + pre)
        out.backward(normal(63, n, H, D, dtype=BF))
        for t in (out, *(t.grad for t in x)):
            assert not t[:pre].any() and not t[mid.stop:].any() and t[mid].isfinite().all() and t[mid].any()


def test_a_block_trains_as_by_hand():
    """Norm, projection, rotary positions, attention: every gradient of one backward pass
    on a stream of its own against the calls made by hand."""
    grids, H, D = [(1, 10, 18), (2, 8, 6)], 4, 72
    E = H * D
    pos, c = vp.vision_positions(grids, 2)
    n, sec = pos.shape[1], (18, 18)
    x, w = normal(13, n, E, dtype=BF), normal(14, 3 * E, E, dtype=BF, std=E ** -0.5)
    gamma, beta = normal(15, E, dtype=BF, std=0.1, mean=1.0), normal(16, E, dtype=BF, std=0.1)
    dout = normal(17, n, H, D, dtype=BF)
    att = vp.Attention(H, H, D)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q, k, v = (vp.layer_norm(*leaves) @ w.t()).view(n, 3, H, D).unbind(1)
        q, k = vp.rope(q, k, pos[1:], sec, axial=True)
        att.forward(q, k, v, c)[0].backward(dout)
    torch.cuda.synchronize()
    y, mean, rstd = vp.layer_norm(x, gamma, beta, stats=True)
    q, k, v = (y @ w.t()).view(n, 3, H, D).unbind(1)
    q, k = vp.rope(q, k, pos[1:], sec, axial=True)
    out, lse = att.forward(q, k, v, c)
    dq, dk, dv = att.backward(dout, q, k, v, out, lse, c)
    dq, dk = vp.rope(dq, dk, pos[1:], sec, axial=True, inverse=True)
    dy = torch.stack([dq, dk, dv], 1).view(n, 3 * E) @ w
    want = vp.layer_norm_backward(dy, x, gamma, mean, rstd)
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


def test_recorded_calls_are_captured():
    """Forward and backward of a block in one graph (no eager graph of its leaves lives),
    replayed on new data."""
    H, D, ql = 2, 64, (100, 30)
    n, c = sum(ql), cu(ql)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    att = vp.Attention(H, H, D)
    x = [normal(20 + i, n, H, D, dtype=BF) for i in range(3)]
    static = [t.clone().requires_grad_() for t in x]

    def step():
        q, k = vp.rope(static[0], static[1], pos, (32,))
        out, _ = att.forward(q, k, static[2], c)
        return [out.detach(), *torch.autograd.grad(out.float().square().sum(), static)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (30, 40):
        with torch.no_grad():
            for i, t in enumerate(static):
                t.copy_(normal(seed + i, n, H, D, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, step()))


def test_outputs_that_are_given():
    H, D, n = 2, 64, 40
    pos, c = torch.ones(1, n, dtype=torch.int32, device=DEV), cu((n,))
    q = normal(50, n, H, D, dtype=BF)
    att = vp.Attention(H, H, D)
    w = torch.ones_like(q).requires_grad_()
    new = lambda: torch.empty_like(q)  # noqa: E731
    for call in (lambda: vp.rope(w, None, pos, (32,), out_q=new()), lambda: vp.rope(q, w, pos, (32,), out_k=new()),
                 lambda: vp.layer_norm(w, out=new()), lambda: att.forward(q, q, w, c, out=new()),
                 lambda: vp.rope(q, None, pos, (32,), out_q=w)):
        with pytest.raises(ValueError, match="output tensors"):
            call()
    with torch.no_grad():
        vp.rope(w, None, pos, (32,), out_q=new())                           # not recorded: taken
    out, lse = att.forward(q, q, q, c)
    mean, rstd = vp.layer_norm(q, stats=True)[1:]
    for write in (lambda t: vp.rope(q, None, pos, (32,), out_q=t), lambda t: vp.rope(q, q, pos, (32,), out_k=t),
                  lambda t: vp.layer_norm(q, out=t), lambda t: vp.layer_norm_backward(q, q, None, mean, rstd, out=t),
                  lambda t: att.forward(q, q, q, c, out=t), lambda t: att.backward(q, q, q, q, out, lse, c, dk=t)):
        t = q.clone()
        loss = (t * w).sum()                                                # saves t
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
