"""Vision-tower operators where element offsets pass 2^31 and 2^32: far rows of large
tensors and of widely strided ones give what the same rows give in small tensors.
About 11 GB on the device at most."""
from __future__ import annotations

import pytest
import torch

import vlm_vision_patch_b200 as vp
from tests.test_gpu_tower import BF, DEV, U, _attention_error_words, attention_ref, close, cu, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("causal,ql", [(False, (40, 90)), (True, (130, 300)), (True, (1, 2))])
def test_attention_on_far_rows(causal, ql):
    """q, k, v and dout share rows of 16384 elements; the sequences are the last of 300000
    rows, 4.9e9 elements in.  Gradients go to rows as wide."""
    D, Hq, Hkv, N, W = 128, 4, 2, 300_000, 16384
    kl = (2500, 700) if ql == (1, 2) else (333, 512)
    nq, nk = sum(ql), sum(kl)
    wide = torch.empty(N, W, dtype=BF, device=DEV)
    part = lambda at, heads: wide[:, at:at + heads * D].view(N, heads, D)  # noqa: E731
    q, k, v, do, out = part(0, Hq), part(1024, Hkv), part(2048, Hkv), part(4096, Hq), part(8192, Hq)
    dq, dk, dv = part(9216, Hq), part(10240, Hkv), part(11264, Hkv)
    small = [normal(70 + i, n, h, D, dtype=BF) for i, (n, h) in enumerate(((nq, Hq), (nk, Hkv), (nk, Hkv), (nq, Hq)))]
    for t, s in zip((q, k, v, do), small):
        t[N - len(s):] = s
    for t in (out, dq, dk, dv):
        t[N - 2000:N] = 5.0
    cq, ck = cu(ql) + (N - nq), cu(kl) + (N - nk)
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    _, lse = att.forward(q, k, v, cq, ck, out=out)
    att.backward(do, q, k, v, out, lse, cq, ck, dq=dq, dk=dk, dv=dv)
    R, A = attention_ref(*small[:3], ql, kl, causal, D ** -0.5, small[3])
    for t, n, m in ((out, "out", nq), (dq, "dq", nq), (dk, "dk", nk), (dv, "dv", nk)):
        close(t[N - m:], R[n], A[n] + U[BF] * R[n].abs() + 1e-30, n)
        if m < 2000:
            assert (t[N - 2000:N - m] == 5).all(), n
    assert ((lse[:, N - nq:].double() - R["lse"]).abs() <= 2.0 ** -15 * (1 + R["lse"].abs())).all()


def test_layer_norm_and_rope_on_far_rows():
    N, E = 270_000, 16384                               # 4.4e9 elements
    x = torch.zeros(N, E, dtype=BF, device=DEV)
    rows = normal(80, 37, E, dtype=BF)
    x[-37:] = rows
    g = normal(81, E, dtype=BF, mean=1.0)
    y, mean, rstd = vp.layer_norm(rows, g, None, stats=True)
    dx, dg, db = vp.layer_norm_backward(rows, rows, g, mean, rstd)
    _, m, r = vp.layer_norm(x, g, None, out=x, stats=True)
    assert torch.equal(x[-37:], y) and torch.equal(m[-37:], mean) and torch.equal(r[-37:], rstd)
    x[-37:] = rows
    x[:-37] = 0
    vp.layer_norm_backward(x, x, g, m, r, out=x)
    assert torch.equal(x[-37:], dx)
    H, D = 64, 256                                      # the same elements as rows of heads
    q, pos = x.view(N, H, D), torch.arange(N, dtype=torch.int32, device=DEV)[None]
    q[-37:] = rows.view(37, H, D)
    vp.rope(q, None, pos, (100,), out_q=q)
    want, _ = vp.rope(rows.view(37, H, D), None, pos[:, -37:].contiguous(), (100,))
    assert torch.equal(q[-37:], want)
