"""Vision-tower operators where inputs are extreme: scores and masked places that
are not finite, sharp rows, rows of no sequence, buffers with guards around them,
and layer-norm sizes whose row ring goes round several times.

References are in 64 bits; tolerances count roundings (U is half a step of the
stored type) and the terms written beside them."""
from __future__ import annotations

import math

import pytest
import torch

import vlm_vision_patch_b200 as vp
from vlm_vision_patch_b200 import _binding as B
from tests.test_gpu_tower import (BF, DEV, F32, F64, SUM, U, _attention_error_words, attention_ref, close, cu,  # noqa: F401
                                  norm_ref, norm_tol, normal, run_attention)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scores of -inf


@pytest.mark.parametrize("D,Hq,Hkv,ql,kl", [
    (64, 2, 2, (300,), (256,)),                 # tiles that no row's end cuts
    (80, 3, 3, (200, 5), (224, 448)),
    (128, 2, 2, (130,), (400,)),
    (64, 16, 16, (64,) * 12, (64,) * 12),       # blocks of one tile, two a multiprocessor
    (96, 24, 24, (100,) * 4, (192,) * 4),
    (128, 12, 2, (1, 2), (9000, 5120)),         # heads packed, the key axis divided and joined
    (64, 8, 8, (1,), (8192,)),
])
def test_rows_whose_every_score_is_minus_infinity(D, Hq, Hkv, ql, kl):
    """exp(-inf - -inf): such a row's output is NaN and its lse -inf, whatever the tiles
    and parts, where a row that sees no key has 0.  Rows with one finite score among
    the infinite ones give that key's value."""
    nq, nk = sum(ql), sum(kl)
    q, k, v = normal(1, nq, Hq, D, dtype=BF), normal(2, nk, Hkv, D, dtype=BF), normal(3, nk, Hkv, D, dtype=BF)
    q[..., 0] = 0
    q[0, :, 0] = 3e38                            # with -3e38 the product overflows to -inf
    k[..., 0] = -3e38
    out, lse = vp.Attention(Hq, Hkv, D).forward(q, k, v, cu(ql), cu(kl))
    assert out[0].isnan().all() and torch.isneginf(lse[:, 0]).all()
    assert out[1:].isfinite().all() and lse[:, 1:].isfinite().all()
    one = kl[0] - 3
    k[one, :, 0] = 0
    out, lse = vp.Attention(Hq, Hkv, D).forward(q, k, v, cu(ql), cu(kl))
    share = Hq // Hkv
    want = v[one].repeat_interleave(share, 0)
    assert torch.equal(out[0], want)
    s = (q[0].double() * k[one].double().repeat_interleave(share, 0)).sum(-1) * D ** -0.5
    # D products in fp32, their sum's and lse's roundings
    tol = D * 2.0 ** -23 * (q[0].double().abs() * k[one].double().repeat_interleave(share, 0).abs()).sum(-1) + 2.0 ** -22
    close(lse[:, 0], s, tol, "lse")


# ------------------------------------------------------------------ masked places that are not finite


CAUSAL = [
    # D, Hq, Hkv, query lengths, key lengths, poisoned (sequence, row from its end)
    (80, 2, 2, (700,), (700,), (0, 401)),
    (64, 2, 1, (300, 515), (300, 515), (1, 130)),
    (128, 4, 2, (513,), (600,), (0, 77)),
    (96, 1, 1, (200,), (130,), (0, 60)),                      # early rows see no key
    (72, 20, 20, (128, 100, 191, 65), (128, 100, 191, 65), (2, 100)),   # blocks of one tile
    (128, 12, 2, (2, 3), (5000, 3000), (1, 1)),               # heads packed, the key axis divided
    (64, 8, 8, (2,), (6000,), (0, 1)),
    (8, 1, 1, (140,), (140,), (0, 7)),
]


@pytest.mark.parametrize("where,value", [("k", math.nan), ("v", math.nan), ("v", math.inf), ("v", -math.inf), ("q", math.nan),
                                         ("do", math.nan), ("do", math.inf), ("q", math.inf)])
@pytest.mark.parametrize("D,Hq,Hkv,ql,kl,at", CAUSAL)
def test_causal_rows_do_not_see_later_rows(D, Hq, Hkv, ql, kl, at, where, value):
    """A NaN or an infinity in a row that the mask hides reaches no result: neither the
    outputs and gradients of earlier queries (from a key or value) nor the gradients
    of later keys (from a query or its gradient)."""
    nq, nk = sum(ql), sum(kl)
    q, do = normal(10, nq, Hq, D, dtype=BF), normal(13, nq, Hq, D, dtype=BF)
    k, v = normal(11, nk, Hkv, D, dtype=BF), normal(12, nk, Hkv, D, dtype=BF)
    R, A = attention_ref(q, k, v, ql, kl, True, D ** -0.5, do)
    s, back = at
    q0, k0, lq, lk = sum(ql[:s]), sum(kl[:s]), ql[s], kl[s]
    x = {"q": q, "k": k, "v": v, "do": do}[where]
    t = (lk if where in "kv" else lq) - back
    c = min(2, D // 8)
    x[(k0 if where in "kv" else q0) + t, :, 5 * c:5 * c + 1] = value       # one element of every head
    got = run_attention(vp.Attention(Hq, Hkv, D, causal=True), q, k, v, do, cu(ql), cu(kl))
    # rows of this sequence that see the poisoned one: queries from `first` on, keys before `last`
    if where in ("k", "v"):
        first, last = max(t - (lk - lq), 0), lk if where == "k" else lk
    else:
        first, last = lq, min(t + lk - lq + 1, lk)
    rows = torch.ones(nq, dtype=torch.bool, device=DEV)
    cols = torch.ones(nk, dtype=torch.bool, device=DEV)
    if where in ("k", "v"):
        rows[q0 + first:q0 + lq] = False
    else:
        rows[q0 + t] = False
    cols[k0:k0 + last] = False
    assert rows.any()
    for n, keep in (("out", rows), ("dq", rows), ("dk", cols), ("dv", cols)):
        if keep.any():
            close(got[n][keep], R[n][keep], A[n][keep] + U[BF] * R[n][keep].abs() + 1e-30, n)
    if where == "do":
        close(got["out"], R["out"], A["out"] + U[BF] * R["out"].abs(), "out")
    # ... and who sees it is not spared
    if where == "v":
        hit = got["out"][q0 + first:q0 + lq, :, 5 * c]
        assert not hit.isfinite().any()
    if where == "do":
        assert not got["dv"][k0:k0 + last, :, 5 * c].isfinite().any()
    if math.isnan(value) and where == "q":
        assert got["out"][q0 + t].isnan().all() and got["dk"][k0:k0 + last].isnan().all()


@pytest.mark.parametrize("D,Hq,Hkv,ql,kl", [(96, 1, 1, (200,), (130,)), (8, 2, 1, (1, 18), (1, 5)), (128, 6, 1, (30, 392), (30, 277))])
def test_causal_rows_without_keys_stay_zero(D, Hq, Hkv, ql, kl):
    """Early rows of a sequence with fewer keys see none: 0 out and 0 gradient, whatever the
    keys of their tile hold."""
    nq, nk = sum(ql), sum(kl)
    q, do = normal(14, nq, Hq, D, dtype=BF), normal(19, nq, Hq, D, dtype=BF)
    k, v = normal(24, nk, Hkv, D, dtype=BF), normal(25, nk, Hkv, D, dtype=BF)
    lo, free = nq - ql[-1], ql[-1] - kl[-1]
    first = nk - kl[-1]
    k[first + 2:], v[first + 2:] = math.nan, math.inf
    got = run_attention(vp.Attention(Hq, Hkv, D, causal=True), q, k, v, do, cu(ql), cu(kl))
    none = slice(lo, lo + free)
    assert not got["out"][none].any() and not got["dq"][none].any() and torch.isneginf(got["lse"][:, none]).all()
    assert got["dq"][none.stop:none.stop + 2].isfinite().all() and got["dq"][none.stop + 2:].isnan().all()


# ------------------------------------------------------------------ values that are not finite, seen


@pytest.mark.parametrize("D,Hq,Hkv,ql,causal", [(80, 2, 2, (300, 70), False), (64, 4, 2, (257,), True), (128, 2, 1, (200, 90), True),
                                                (96, 2, 2, (130,), False)])
def test_dv_does_not_depend_on_v(D, Hq, Hkv, ql, causal):
    """dv_j = sum_i p_ij dout_i: a NaN in v makes out, dq and dk NaN (through delta), and
    dv is what it was; an infinite element of dout reaches its own column of dv only."""
    n = sum(ql)
    q, do = normal(15, n, Hq, D, dtype=BF), normal(18, n, Hq, D, dtype=BF)
    k, v = normal(16, n, Hkv, D, dtype=BF), normal(17, n, Hkv, D, dtype=BF)
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    clean = run_attention(att, q, k, v, do, cu(ql), cu(ql))
    bad = v.clone()
    bad[3, :, 1] = math.nan
    got = run_attention(att, q, k, bad, do, cu(ql), cu(ql))
    assert torch.equal(got["dv"], clean["dv"]) and torch.equal(got["lse"], clean["lse"])
    seen = slice(3 if causal else 0, ql[0])
    assert got["out"][seen, :, 1].isnan().all() and got["dq"][seen].isnan().all()
    assert not got["dk"][:ql[0]].isfinite().any()
    for x in ("out", "dq", "dk"):
        assert torch.equal(got[x][ql[0]:], clean[x][ql[0]:])
    bad = do.clone()
    bad[ql[0] - 1, :, 2] = math.inf                       # the row that sees every key
    got = run_attention(att, q, k, v, bad, cu(ql), cu(ql))
    other = [d for d in range(D) if d != 2]
    assert torch.equal(got["dv"][..., other], clean["dv"][..., other])
    assert (got["dv"][:ql[0], :, 2] == math.inf).all() and not got["dk"][:ql[0]].isfinite().any()


# ------------------------------------------------------------------ rows of no sequence


@pytest.mark.parametrize("D,Hq,Hkv,causal,pre,ql,kl,post", [
    (80, 2, 2, False, 0, (130, 61), None, 200),
    (64, 2, 1, True, 7, (300, 0, 45), None, 19),
    (128, 12, 2, True, 3, (1, 1), (5000, 3000), 2),           # divided keys, packed heads
    (72, 20, 20, False, 0, (64,) * 12, None, 700),            # blocks of one tile
    (96, 2, 2, False, 5, (0, 0), None, 4),                    # every sequence empty
    (96, 2, 2, False, 5, (), None, 4),                        # no sequence
    (128, 12, 2, True, 100, (200,), (300,), 3000),            # dk and dv in parts
])
def test_padded_batches_in_tensors_that_hold_zeros(D, Hq, Hkv, causal, pre, ql, kl, post):
    """Rows before the first and behind the last sequence keep what given tensors held,
    in every form of the kernels, whatever the inputs hold there."""
    kl = ql if kl is None else kl
    nq, nk = pre + sum(ql) + post, pre + sum(kl) + post
    q, do = normal(30, nq, Hq, D, dtype=BF), normal(33, nq, Hq, D, dtype=BF)
    k, v = normal(31, nk, Hkv, D, dtype=BF), normal(32, nk, Hkv, D, dtype=BF)
    mq, mk = slice(pre, pre + sum(ql)), slice(pre, pre + sum(kl))
    R, A = attention_ref(q[mq], k[mk], v[mk], ql, kl, causal, D ** -0.5, do[mq])
    for t, m in ((q, mq), (do, mq), (k, mk), (v, mk)):
        t[:m.start], t[m.stop:] = math.nan, math.inf
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    cq, ck = cu(ql) + pre, cu(kl) + pre
    out, lse = att.forward(q, k, v, cq, ck, out=torch.zeros_like(q))
    dq, dk, dv = att.backward(do, q, k, v, out, lse, cq, ck, dq=torch.zeros_like(q), dk=torch.zeros_like(k),
                              dv=torch.zeros_like(v))
    for t, n, m in ((out, "out", mq), (dq, "dq", mq), (dk, "dk", mk), (dv, "dv", mk)):
        assert not t[:m.start].any() and not t[m.stop:].any(), n
        close(t[m], R[n], A[n] + U[BF] * R[n].abs() + 1e-30, n)


# ------------------------------------------------------------------ sharp rows


def sharp_tolerances(q, k, v, do, ql, scale, dq2):
    """References of one-head-per-key attention (no mask) and tolerances element by
    element.  With T_ij = D 2^-23 scale sum_d |q||k| (a score's error: D products and
    additions in fp32, truncated) a row's lse is off by sum_j p_ij T_ij + 2^-22 (1 + |lse|)
    (its own and its product's rounding), and the recomputed p by a factor exp of both
    (and 2^-22 |s| of the exponent's rounding; 2^-12 covers what is second order).  ds = p (dp - delta) takes that error,
    dp's fp32 sum, delta's and its own rounding to bf16.  `dq2`: rows of at most 256
    keys take delta from the recomputed p and dp, the others from the stored output."""
    R = {n: torch.zeros_like(t, dtype=F64) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    A = {n: torch.zeros_like(t) for n, t in R.items()}
    u, D, i = U[BF], q.shape[-1], 0
    q, k, v, do = (t.double() for t in (q, k, v, do))
    for m in ql:
        for h in range(q.shape[1]):
            qs, ks, vs, g = (t[i:i + m, h] for t in (q, k, v, do))
            s = qs @ ks.t() * scale
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - lse)
            T = D * 2.0 ** -23 * scale * (qs.abs() @ ks.abs().t())
            e = torch.expm1(T + (p * T).sum(1, keepdim=True) + 2.0 ** -22 * (1 + lse.abs() + s.abs())) + 2.0 ** -12
            o, dp = p @ vs, g @ vs.t()
            ao = ((u + e) * p) @ vs.abs()
            dpe = D * 2.0 ** -23 * (g.abs() @ vs.abs().t())
            delta = (g * o).sum(1, keepdim=True)
            if dq2 and m <= 256:
                de = (p * (e * (dp - delta).abs() + dpe)).sum(1, keepdim=True) + (p * e).sum(1, keepdim=True) * (
                    g.abs() * (u * o.abs() + ao)).sum(1, keepdim=True) + 2.0 ** -20 * (g.abs() * o.abs()).sum(1, keepdim=True)
            else:
                de = (g.abs() * (u * o.abs() + ao)).sum(1, keepdim=True) + D * 2.0 ** -23 * (g.abs() * o.abs()).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dse = (u + e) * ds.abs() + p * (1 + e) * (dpe + de)
            x = slice(i, i + m)
            R["out"][x, h], A["out"][x, h] = o, ao
            R["dv"][x, h], A["dv"][x, h] = p.t() @ g, ((u + e) * p).t() @ g.abs()
            R["dq"][x, h], A["dq"][x, h] = scale * (ds @ ks), scale * (dse @ ks.abs())
            R["dk"][x, h], A["dk"][x, h] = scale * (ds.t() @ qs), scale * (dse.t() @ qs.abs())
        i += m
    return R, {n: A[n] + u * R[n].abs() + 1e-30 for n in R}


@pytest.mark.parametrize("D,std", [(80, 0.05), (80, 1.0), (80, 4.0), (80, 16.0), (128, 4.0), (64, 16.0)])
def test_attention_gradients_from_flat_to_one_hot(D, std):
    H, ql = 2, (700, 90, 200)
    n = sum(ql)
    q, k = normal(20, n, H, D, dtype=BF, std=std), normal(21, n, H, D, dtype=BF, std=std)
    k[::7] *= 3
    v, do = normal(22, n, H, D, dtype=BF), normal(23, n, H, D, dtype=BF)
    got = run_attention(vp.Attention(H, H, D), q, k, v, do, cu(ql), cu(ql))
    R, A = sharp_tolerances(q, k, v, do, ql, D ** -0.5, True)
    for name in ("out", "dv", "dq", "dk"):
        close(got[name], R[name], A[name], name)
        # the tolerance tells a gradient from none, and so from the wrong sign: nearly everywhere while
        # rows share their weight, on the rows with two close scores where they are one-hot
        told = (R[name].abs() > A[name]).double()
        assert told.mean() > 0.1 if std < 16 else told.sum() >= 100, name


# ------------------------------------------------------------------ buffers with guards


class Guards:
    """Tensors inside larger allocations whose other elements must not change."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=BF):
        n, pad = math.prod(shape), 4096
        flat = torch.full((n + 2 * pad,), 77.0, dtype=dtype, device=DEV)
        self.all.append((flat, n, pad))
        return flat[pad:pad + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for flat, n, pad in self.all:
            assert (flat[:pad] == 77).all() and (flat[pad + n:] == 77).all()


def heads(t):
    return B.pe_heads(t.data_ptr(), t.stride(0), t.stride(1))


@pytest.mark.parametrize("D,Hq,Hkv,causal,nq,nk,cq,ck", [
    (64, 1, 1, False, 300, 300, (-5, 100, 60, 5000), None),
    (80, 4, 2, True, 300, 300, (-5, 100, 60, 5000), None),
    (72, 2, 2, False, 131, 200, (0, 50, 131), (-2 ** 31, 2 ** 31 - 1, 3)),
    (128, 12, 2, True, 4, 9000, (0, 1, 9, 2), (0, 9001, 4000, 20000)),     # packed and divided
    (64, 8, 8, False, 2, 6000, (-1, 1, 7), (0, 6500, 100)),
    (96, 24, 24, True, 500, 500, (3, 70, 130, 190, 250, 64, 330, 400, 999), None),
    (128, 4, 2, True, 513, 700, (0, 513), (0, 700)),                       # in order, for comparison
    (40, 2, 2, False, 77, 77, (77, 0), (0, 77)),
])
def test_nothing_outside_the_buffers_is_written(D, Hq, Hkv, causal, nq, nk, cq, ck):
    """Outputs, gradients, lse and both workspaces between guards, boundaries in and out
    of their contract."""
    G = Guards()
    c1 = torch.tensor(cq, dtype=torch.int32, device=DEV)
    c2 = c1 if ck is None else torch.tensor(ck, dtype=torch.int32, device=DEV)
    n = len(cq) - 1
    q, do = normal(40, nq, Hq, D, dtype=BF), normal(43, nq, Hq, D, dtype=BF)
    k, v = normal(41, nk, Hkv, D, dtype=BF), normal(42, nk, Hkv, D, dtype=BF)
    out, dq, dk, dv = G(nq, Hq, D), G(nq, Hq, D), G(nk, Hkv, D), G(nk, Hkv, D)
    lse = G(Hq, nq, dtype=F32)
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    ws = [G(max(B.pe_attention_workspace(att.h, n, nq, nk, b), 16) // 4, dtype=F32) for b in (False, True)]
    st = torch.cuda.current_stream().cuda_stream
    B.pe_attention_forward(att.h, n, c1.data_ptr(), nq, c2.data_ptr(), nk, heads(q), heads(k), heads(v), heads(out),
                           lse.data_ptr(), ws[0].data_ptr(), ws[0].numel() * 4, st)
    B.pe_attention_backward(att.h, n, c1.data_ptr(), nq, c2.data_ptr(), nk, heads(q), heads(k), heads(v), heads(out),
                            lse.data_ptr(), heads(do), heads(dq), heads(dk), heads(dv), ws[1].data_ptr(), ws[1].numel() * 4, st)
    G.check()
    if cq[0] == -5:                                        # rows 0 .. 59 belong to the first sequence, of 100 rows, alone
        R, A = attention_ref(q[:100], k[:100], v[:100], (100,), (100,), causal, D ** -0.5, do[:100])
        for got, x in ((out, "out"), (dq, "dq")):
            close(got[:60], R[x][:60], A[x][:60] + U[BF] * R[x][:60].abs() + 1e-30, x)
    # the same through the wrapper, whose tensors are its own
    att.forward(q, k, v, c1, c2)
    att.backward(do, q, k, v, out, lse, c1, c2)
    G.check()


# ------------------------------------------------------------------ layer norm


@pytest.mark.parametrize("N,E,dtype", [
    # threads a row, chunks a thread: 32 x 5, 64 x 3, 64 x 4, 128 x 4, 256 x 4, 256 x 5, 512 x 4
    (8003, 1280, BF), (3001, 1288, BF), (3001, 2048, BF), (2005, 4096, BF), (1301, 8192, BF), (701, 10240, BF), (701, 16384, BF),
    (8003, 640, F32), (3001, 1152, F32), (3001, 1280, F32), (2005, 2560, F32), (1301, 4096, F32), (701, 5120, F32),
    (701, 8192, F32), (701, 16384, F32),                      # the last keeps one row in flight
])
def test_layer_norm_backward_over_many_rows(N, E, dtype):
    """More rows than the resident blocks hold at once (three to five times, the last
    group partly empty): ring slots, row sums and weight sums are used again and again."""
    x = normal(50, N, E, dtype=dtype, std=1.5, mean=-0.2)
    g = normal(51, E, dtype=dtype, std=0.2, mean=1.0)
    dy = normal(52, N, E, dtype=dtype)
    _, mean, rstd = vp.layer_norm(x, g, None, 1e-5, stats=True)
    dx, dg, db = vp.layer_norm_backward(dy, x, g, mean, rstd)
    _, _, rr, z = norm_ref(x, g, None, 1e-5)
    d, a = dy.double(), dy.double() * g.double()
    rdx = rr[:, None] * (a - a.mean(-1, keepdim=True) - z * (a * z).mean(-1, keepdim=True))
    tz = norm_tol(x, None, None, 0 * z, x.double().mean(-1), rr, z, F32)
    t = (a.abs() * 4 * 2.0 ** -24 + SUM * a.abs().mean(-1, keepdim=True)
         + tz * (a * z).mean(-1, keepdim=True).abs()
         + z.abs() * (SUM * (a * z).abs().mean(-1, keepdim=True) + (a.abs() * tz).mean(-1, keepdim=True)))
    close(dx, rdx, rr[:, None] * t + 2 * SUM * rdx.abs() + U[dtype] * rdx.abs(), "dx")
    # a column's chain: the rows of one block, its other rows, the 32 x 4 sums over blocks and their join
    chain = (64 + N / 148) * 2.0 ** -24
    rdg, rdb = (d * z).sum(0), d.sum(0)
    close(dg, rdg, (d.abs() * tz).sum(0) + chain * (d * z).abs().sum(0) + U[dtype] * rdg.abs(), "dgamma")
    close(db, rdb, chain * d.abs().sum(0) + U[dtype] * rdb.abs(), "dbeta")
    again = vp.layer_norm_backward(dy, x, g, mean, rstd)
    assert all(torch.equal(p, w) for p, w in zip(again, (dx, dg, db)))
    xi = x.clone()
    assert torch.equal(vp.layer_norm_backward(dy, xi, g, mean, rstd, weight_grads=False, out=xi)[0], dx)
