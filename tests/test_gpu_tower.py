"""Vision-tower operators on a B200 against plain 64-bit implementations: patch
positions, rotary positions, layer norm and attention, with their gradients.

Tolerances count roundings.  U is half a step of the stored type relative to the
value (bf16 2^-8, fp32 2^-24); sums in fp32 get the bounds written beside them.
"""
from __future__ import annotations

import math

import pytest
import torch

import vlm_vision_patch_b200 as vp
from vlm_vision_patch_b200 import PEError
from vlm_vision_patch_b200 import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _attention_error_words(monkeypatch):
    made = []
    orig = vp.Attention.__init__

    def init(self, *a, **k):
        orig(self, *a, **k)
        made.append(self)
    monkeypatch.setattr(vp.Attention, "__init__", init)
    yield
    torch.cuda.synchronize()
    for a in made:
        assert a.last_error() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(seed, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * std + mean).to(dtype)


def close(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; first {i}: got "
                             f"{float(got[i])}, expected {float(ref[i])} +- {float(torch.as_tensor(tol).expand_as(err)[i])}")


# ------------------------------------------------------------------ positions


def positions_ref(grids, m):
    rows, cu = [], [0]
    for t, h, w in grids:
        for f in range(t):
            for wr in range(h // m):
                for wc in range(w // m):
                    for a in range(m):
                        for b in range(m):
                            rows.append((f, wr * m + a, wc * m + b))
            cu.append(cu[-1] + h * w)
    return torch.tensor(rows, dtype=torch.int32).reshape(-1, 3).t(), torch.tensor(cu, dtype=torch.int32)


@pytest.mark.parametrize("grids,m", [
    ([(1, 16, 64)], 2), ([(4, 14, 14)], 2), ([(1, 1, 1)], 1), ([(3, 5, 7), (1, 2, 9)], 1), ([(2, 6, 9), (1, 3, 3)], 3),
    ([(1, 4, 8)], 4), ([(1, 2, 2)] * 64, 2), ([(1 + i % 3, 2, 2 + 2 * (i % 5)) for i in range(150)], 2), ([], 2),
])
def test_positions(grids, m):
    pos, cu = vp.vision_positions(grids, m)
    rp, rc = positions_ref(grids, m)
    assert torch.equal(pos.cpu(), rp) and torch.equal(cu.cpu(), rc)


def test_positions_follow_the_patch_order():
    """The same order as the forward calls' rows: frames that hold their own
    (row, column) patchify into rows with these positions."""
    p, m, h, w = 14, 2, 6, 8
    pe = vp.PatchEmbed(64, 1, 1, p)
    yy = torch.arange(h, device=DEV, dtype=F32).repeat_interleave(p)[:, None].expand(h * p, w * p)
    xx = torch.arange(w, device=DEV, dtype=F32).repeat_interleave(p)[None].expand(h * p, w * p)
    frames = torch.stack([yy, xx])[:, None].contiguous()          # frame 0: rows, frame 1: columns
    rows = pe.patchify([frames], [(2, h, w)], m, rows_dtype=F32)
    pos, cu = vp.vision_positions([(2, h, w)], m)
    n = h * w
    assert torch.equal(rows[:n, 0].int(), pos[1, :n]) and torch.equal(rows[n:, 0].int(), pos[2, n:])
    assert cu.tolist() == [0, n, 2 * n]


# ------------------------------------------------------------------ rotary positions


def rope_ref(x, pos, sections, theta, axial, sign):
    S = sum(sections)
    rate = torch.cat([torch.tensor([theta ** (-(j / n if axial else (j + sum(sections[:a])) / S)) for j in range(n)],
                                   dtype=F64) for a, n in enumerate(sections)]).to(x.device)
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=x.device)
    ang = pos.double()[axis].t() * rate * sign
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x = x.double()
    a, b = x[..., :S], x[..., S:2 * S]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * S:]], -1)


def rope_tol(x, ref, S, dtype):
    """|a| + |b| times the error of a cosine in fp32 (the angle's fraction of a turn
    is rounded to 2^-25 of a turn at most, 2 pi 2^-25 < 2^-22, sincospif and the
    products add a few 2^-24): 2^-21; then the stored rounding."""
    x = x.double().abs()
    both = x[..., :S] + x[..., S:2 * S]
    return torch.cat([both, both, 0 * x[..., 2 * S:]], -1) * 2.0 ** -21 + ref.abs() * U[dtype]


ROPE = [
    # N, Hq, Hk, D, sections, axial, theta, far
    (1024, 16, 16, 80, (20, 20), True, 1e4, 96),
    (513, 3, 2, 72, (18, 18), True, 1e4, 96),
    (257, 12, 2, 128, (16, 24, 24), False, 1e6, 1 << 20),
    (1, 1, 1, 2, (1,), False, 1e4, 5),
    (7, 2, 1, 96, (12, 10, 10), False, 1e4, 10000),         # a tail that is copied
    (9, 1, 3, 22, (0, 3, 0, 4), True, 100.0, 1000),         # empty sections, odd sizes
    (64, 5, 0, 256, (128,), False, 1e4, 2 ** 31 - 1),       # no keys, the widest turn, the farthest position
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,D,sections,axial,theta,far", ROPE)
def test_rope(N, Hq, Hk, D, sections, axial, theta, far, inverse, dtype):
    q = normal(1, N, Hq, D, dtype=dtype)
    k = normal(2, N, Hk, D, dtype=dtype) if Hk else None
    pos = torch.randint(0, far, (len(sections), N), generator=gen(3), device=DEV, dtype=torch.int64).int()
    oq, ok = vp.rope(q, k, pos, sections, theta, axial, inverse)
    for x, o in ((q, oq), (k, ok)):
        if x is None:
            assert o is None
            continue
        ref = rope_ref(x, pos, sections, theta, axial, -1.0 if inverse else 1.0)
        close(o, ref, rope_tol(x, ref, sum(sections), dtype), "rope")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [80, 72, 34, 30])
def test_rope_strides_and_in_place(D, dtype):
    """Slices of a packed projection, a base that is not 16-byte aligned, and in
    place: the same bits as dense tensors."""
    N, H = 133, 4
    pos = torch.randint(0, 99, (2, N), generator=gen(5), device=DEV, dtype=torch.int32)
    sec = (D // 4, D // 4)
    flat = normal(6, 1 + N * 3 * H * D, dtype=dtype)
    qkv = flat[1:].view(N, 3, H, D)
    q, k = qkv[:, 0], qkv[:, 1]
    dq, dk = vp.rope(q.contiguous(), k.contiguous(), pos, sec, axial=True)
    sq, sk = vp.rope(q, k, pos, sec, axial=True)
    assert torch.equal(dq, sq) and torch.equal(dk, sk)
    v = qkv[:, 2].clone()
    iq, ik = vp.rope(q, k, pos, sec, axial=True, out_q=q, out_k=k)
    assert iq.data_ptr() == q.data_ptr() and torch.equal(iq, dq) and torch.equal(ik, dk) and torch.equal(qkv[:, 2], v)
    hq = q.transpose(0, 1).contiguous().transpose(0, 1)          # heads outermost
    bq, _ = vp.rope(hq, None, pos, sec, axial=True, inverse=True)
    assert torch.equal(bq, vp.rope(dq, None, pos, sec, axial=True, inverse=True)[0])


def test_rope_gradient_is_the_transpose():
    """<rope(x), w> = <x, rope^-1(w)>, up to the roundings of both sides."""
    N, H, D = 300, 2, 64
    pos = torch.randint(0, 500, (3, N), generator=gen(7), device=DEV, dtype=torch.int32)
    x, w = normal(8, N, H, D), normal(9, N, H, D)
    y, _ = vp.rope(x, None, pos, (8, 12, 12))
    g, _ = vp.rope(w, None, pos, (8, 12, 12), inverse=True)
    a, b = (y.double() * w.double()).sum(), (x.double() * g.double()).sum()
    assert abs(float(a - b)) <= 2.0 ** -20 * float((x.double().abs() * 2 * w.double().abs().amax()).sum())


def test_rope_empty():
    q = torch.empty(0, 2, 8, device=DEV)
    oq, ok = vp.rope(q, q, torch.empty(1, 0, dtype=torch.int32, device=DEV), (4,))
    assert oq.shape == (0, 2, 8) and ok.shape == (0, 2, 8)


# ------------------------------------------------------------------ layer norm


def norm_ref(x, g, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = (x - mean).square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    z = (x - mean) * rstd
    y = z
    if g is not None:
        y = y * g.double()
    if b is not None:
        y = y + b.double()
    return y, mean[..., 0], rstd[..., 0], z


# at most 5 * 8 + 4 additions follow one another in a row's sums, and 16 warps': 64 roundings cover a statistic
SUM = 64 * 2.0 ** -24


def norm_tol(x, g, b, y, mean, rstd, z, dtype):
    """mean is off by SUM mean|x|, rstd by SUM relative (and by the mean's error,
    second order in the deviations); z inherits both."""
    off = rstd[..., None] * SUM * x.double().abs().mean(-1, keepdim=True)
    tz = off + (SUM + off.square()) * z.abs() + 2.0 ** -22 * rstd[..., None] * x.double().abs()
    ga = 1.0 if g is None else g.double().abs()
    return ga * tz + U[dtype] * y.abs() + 2.0 ** -22 * (0 if b is None else b.double().abs())


NORM = [(1, 8), (5, 64), (1024, 1280), (33, 1152), (7, 1288), (3, 2048), (130, 1000), (5, 4096), (2, 4104), (3, 8192),
        (2, 16384), (257, 256)]


@pytest.mark.parametrize("w_dtype", [BF, F32, None])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,E", NORM)
def test_layer_norm(N, E, dtype, w_dtype):
    x = normal(10, N, E, dtype=dtype, std=2.0, mean=0.5)
    g = None if w_dtype is None else normal(11, E, dtype=w_dtype, std=0.2, mean=1.0)
    b = None if w_dtype is None else normal(12, E, dtype=w_dtype, std=0.2)
    y, mean, rstd = vp.layer_norm(x, g, b, 1e-6, stats=True)
    ry, rm, rr, rz = norm_ref(x, g, b, 1e-6)
    close(mean, rm, SUM * x.double().abs().mean(-1), "mean")
    close(rstd, rr, 2 * SUM * rr, "rstd")
    close(y, ry, norm_tol(x, g, b, ry, rm, rr, rz, dtype), "y")
    assert torch.equal(vp.layer_norm(x, g, b, 1e-6), y)
    xi = x.clone()
    assert vp.layer_norm(xi, g, b, 1e-6, out=xi) is xi and torch.equal(xi, y)


@pytest.mark.parametrize("w_dtype", [BF, F32, None])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,E", NORM + [(5000, 64)])
def test_layer_norm_backward(N, E, dtype, w_dtype):
    x = normal(13, N, E, dtype=dtype, std=1.5, mean=-0.2)
    g = None if w_dtype is None else normal(14, E, dtype=w_dtype, std=0.2, mean=1.0)
    dy = normal(15, N, E, dtype=dtype)
    _, mean, rstd = vp.layer_norm(x, g, None, 1e-5, stats=True)
    dx, dg, db = vp.layer_norm_backward(dy, x, g, mean, rstd)
    _, _, rr, z = norm_ref(x, g, None, 1e-5)
    d, a = dy.double(), dy.double() * (1.0 if g is None else g.double())
    rdx = rr[:, None] * (a - a.mean(-1, keepdim=True) - z * (a * z).mean(-1, keepdim=True))
    wt = w_dtype or F32
    assert dg.dtype == db.dtype == wt
    # z itself is off by tz; the row's two means by SUM of their absolute terms
    tz = norm_tol(x, None, None, 0 * z, x.double().mean(-1), rr, z, F32)
    t = (a.abs() * 4 * 2.0 ** -24 + SUM * a.abs().mean(-1, keepdim=True)
         + tz * (a * z).mean(-1, keepdim=True).abs()
         + z.abs() * (SUM * (a * z).abs().mean(-1, keepdim=True) + (a.abs() * tz).mean(-1, keepdim=True)))
    close(dx, rdx, rr[:, None] * t + 2 * SUM * rdx.abs() + U[dtype] * rdx.abs(), "dx")
    # a column: at most N/4 + 4 + N/8 additions in one chain, far fewer once blocks share it
    chain = (64 + N / 148) * 2.0 ** -24
    rdg, rdb = (d * z).sum(0), d.sum(0)
    close(dg, rdg, (d.abs() * tz).sum(0) + chain * (d * z).abs().sum(0) + U[wt] * rdg.abs(), "dgamma")
    close(db, rdb, chain * d.abs().sum(0) + U[wt] * rdb.abs(), "dbeta")
    dx2, n1, n2 = vp.layer_norm_backward(dy, x, g, mean, rstd, weight_grads=False)
    assert n1 is None and n2 is None and torch.equal(dx2, dx)
    again = vp.layer_norm_backward(dy, x, g, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dg, db)))
    dyi = dy.clone()
    vp.layer_norm_backward(dyi, x, g, mean, rstd, weight_grads=False, out=dyi)
    assert torch.equal(dyi, dx)


def test_layer_norm_gradient_against_differences():
    """<dx, u> against (f(x + h u) - f(x - h u)) / 2h of the 64-bit forward pass;
    the difference is off by h^2 (below 1e-8) and the kernel by fp32 roundings."""
    N, E, h = 6, 96, 1e-5
    x, dy, u = normal(16, N, E), normal(17, N, E), normal(18, N, E)
    g, b = normal(19, E, mean=1.0, std=0.1), normal(20, E)
    _, mean, rstd = vp.layer_norm(x, g, b, 1e-6, stats=True)
    dx, dg, _ = vp.layer_norm_backward(dy, x, g, mean, rstd)
    f = lambda xx, gg: (norm_ref(xx, gg, b, 1e-6)[0] * dy.double()).sum()  # noqa: E731
    num = (f(x.double() + h * u.double(), g) - f(x.double() - h * u.double(), g)) / (2 * h)
    assert abs(float(num - (dx.double() * u.double()).sum())) <= 1e-5 * float((dx.double() * u.double()).abs().sum())
    w = normal(21, E).double()
    num = (f(x, g.double() + h * w) - f(x, g.double() - h * w)) / (2 * h)
    assert abs(float(num - (dg.double() * w).sum())) <= 1e-5 * float((dg.double() * w).abs().sum())


def test_layer_norm_rows_are_independent():
    """A row of NaN or infinities leaves the other rows' results as they are, and a
    constant row gives beta (its deviations are 0)."""
    x = normal(22, 9, 320)
    y0 = vp.layer_norm(x)
    x2 = x.clone()
    x2[3] = math.nan
    x2[5, 7] = math.inf
    x2[8] = 4.0
    y = vp.layer_norm(x2)
    keep = [0, 1, 2, 4, 6, 7]
    assert torch.equal(y[keep], y0[keep]) and y[3].isnan().all() and y[5].isnan().all() and not y[8].any()


def test_layer_norm_empty():
    x = torch.empty(0, 64, device=DEV)
    y, mean, rstd = vp.layer_norm(x, stats=True)
    dx, dg, db = vp.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == x.shape and not dg.any() and not db.any()


# ------------------------------------------------------------------ attention


def cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(device=DEV, dtype=torch.int32)


def attention_ref(q, k, v, ql, kl, causal, scale, do=None):
    """out, lse, dq, dk, dv in 64 bits, and the sums of absolute terms that their
    tolerances scale with."""
    hq, hk = q.shape[1], k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    R = {n: torch.zeros_like(t) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    A = {n: torch.zeros_like(t) for n, t in R.items()}
    R["lse"] = torch.full((hq, q.shape[0]), -math.inf, device=DEV, dtype=F64)
    E = 2.0 ** -12           # scores: D products in fp32 (2^-24 * 128), exp and sums: far below 2^-12 of a probability
    u = U[BF]
    i = j = 0
    for m, n in zip(ql, kl):
        for h in range(hq):
            hh = h * hk // hq
            qs, ks, vs = q[i:i + m, h], k[j:j + n, hh], v[j:j + n, hh]
            s = qs @ ks.t() * scale
            if causal:
                s = s.masked_fill(torch.arange(n, device=DEV) > torch.arange(m, device=DEV)[:, None] + n - m, -math.inf)
            lse = torch.logsumexp(s, 1) if n else torch.full((m,), -math.inf, device=DEV, dtype=F64)
            p = torch.where(torch.isinf(lse)[:, None], 0.0, torch.exp(s - lse.nan_to_num(0, 0, 0)[:, None]))
            R["lse"][h, i:i + m] = lse
            o = p @ vs
            R["out"][i:i + m, h] = o
            A["out"][i:i + m, h] = (u + E) * (p @ vs.abs())
            if do is not None:
                g = do[i:i + m, h].double()
                ds = p * (g @ vs.t() - (g * o).sum(1, keepdim=True))
                # ds: its own rounding, delta from the stored out (u |do||out| and out's own error), dp in fp32
                dse = (u + E) * ds.abs() + p * ((g.abs() * (u * o.abs() + A["out"][i:i + m, h])).sum(1, keepdim=True)
                                               + E * (g.abs() @ vs.abs().t()))
                R["dv"][j:j + n, hh] += p.t() @ g
                A["dv"][j:j + n, hh] += (u + E) * (p.t() @ g.abs())
                R["dq"][i:i + m, h] = scale * (ds @ ks)
                A["dq"][i:i + m, h] = scale * (dse @ ks.abs())
                R["dk"][j:j + n, hh] += scale * (ds.t() @ qs)
                A["dk"][j:j + n, hh] += scale * (dse.t() @ qs.abs())
        i, j = i + m, j + n
    return R, A


def check_attention(got, R, A, nq, nk, names=("out", "dq", "dk", "dv")):
    for n in names:
        rows = nq if n in ("out", "dq") else nk
        close(got[n][:rows], R[n][:rows], A[n][:rows] + U[BF] * R[n][:rows].abs() + 1e-30, n)
    lse, ref = got["lse"][:, :nq].double(), R["lse"][:, :nq]
    assert torch.equal(torch.isinf(lse), torch.isinf(ref))
    fin = ~torch.isinf(ref)
    # scores are off by D 2^-24 of their terms; sums of up to 2^14 keys in fp32 by 2^-16 at most
    assert ((lse - ref)[fin].abs() <= 2.0 ** -15 * (1 + ref[fin].abs())).all()


def run_attention(att, q, k, v, do, cq, ck):
    out, lse = att.forward(q, k, v, cq, ck)
    got = {"out": out, "lse": lse}
    if do is not None:
        got["dq"], got["dk"], got["dv"] = att.backward(do, q, k, v, out, lse, cq, ck)
    return got


SHAPES = [
    # D, Hq, Hkv, query lengths, key lengths (None: the same), causal
    (80, 16, 16, (64,), None, False),
    (80, 2, 2, (196, 196, 196, 196), None, False),
    (72, 3, 3, (1, 127, 128, 129), None, False),
    (64, 2, 1, (255, 256, 257, 2), None, False),
    (128, 4, 2, (300, 0, 17, 513), None, True),
    (128, 12, 2, (1, 1, 1), (1000, 129, 1), True),
    (8, 1, 1, (5, 3), None, False),
    (16, 2, 2, (130,), None, True),
    (40, 2, 1, (70, 200), (333, 5), False),
    (88, 2, 2, (200, 64), (64, 200), True),        # the first sequence's early rows see no key
    (96, 6, 1, (33, 1, 384), (0, 7, 385), False),  # a sequence without keys
    (120, 1, 1, (0, 9, 0, 260), (4, 9, 0, 300), True),
    (80, 2, 2, (1024, 3), None, False),
    (128, 2, 2, (640,), None, True),
    (64, 1, 1, (7,), (2500,), False),
    (80, 1, 1, (2500,), (7,), False),
    (32, 4, 4, tuple([3, 9, 1, 30] * 20), None, False),
    # few rows on long keys: the key axis divided over blocks, heads packed into a tile
    (128, 12, 2, (1, 2, 1), (5000, 3000, 77), True),
    (64, 8, 8, (1, 1), (6000, 4500), False),
    (80, 6, 2, (20, 3, 0), (9000, 4000, 300), False),
    (96, 16, 1, (5,), (7001,), True),
    (128, 2, 1, (1, 40), (0, 9000), False),
    (72, 5, 1, (9, 25, 11), (3100, 2000, 5000), True),
]


@pytest.mark.parametrize("D,Hq,Hkv,ql,kl,causal", SHAPES)
def test_attention(D, Hq, Hkv, ql, kl, causal):
    kl = ql if kl is None else kl
    nq, nk = sum(ql), sum(kl)
    q, do = normal(30, nq, Hq, D, dtype=BF), normal(33, nq, Hq, D, dtype=BF)
    k, v = normal(31, nk, Hkv, D, dtype=BF), normal(32, nk, Hkv, D, dtype=BF)
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    got = run_attention(att, q, k, v, do, cu(ql), cu(kl))
    R, A = attention_ref(q, k, v, ql, kl, causal, D ** -0.5, do)
    check_attention(got, R, A, nq, nk)
    again = run_attention(att, q, k, v, do, cu(ql), cu(kl))
    assert all(torch.equal(got[n], again[n]) for n in got), "two runs differ"
    out, none = att.forward(q, k, v, cu(ql), cu(kl), lse=False)
    assert none is None and torch.equal(out, got["out"])


@pytest.mark.parametrize("std", [0.05, 4.0, 16.0])
def test_attention_sharp_and_flat_scores(std):
    """From nearly uniform to one-hot rows: the running maximum moves by hundreds."""
    D, H, ql = 80, 2, (700, 90)
    n = sum(ql)
    q, k = normal(34, n, H, D, dtype=BF, std=std), normal(35, n, H, D, dtype=BF, std=std)
    k[::7] *= 3
    v, do = normal(36, n, H, D, dtype=BF), normal(37, n, H, D, dtype=BF)
    got = run_attention(vp.Attention(H, H, D), q, k, v, do, cu(ql), cu(ql))
    R, A = attention_ref(q, k, v, ql, ql, False, D ** -0.5, do)
    check_attention(got, R, A, n, n, ("out", "dv"))
    # ds inherits a score's absolute error, 128 * 2^-24 of |q||k| scale: with std 16 up to 2^-17 * 2000 * 3 = 0.05 of p
    smax = float((q.double().abs().amax() * k.double().abs().amax()) * D ** 0.5)
    for name in ("dq", "dk"):
        extra = A[name] / U[BF] * (2.0 ** -17 * smax)
        close(got[name], R[name], A[name] + extra + U[BF] * R[name].abs() + 1e-30, name)


def test_attention_layouts():
    """Packed projections, heads outermost and a packed gradient: the bits of dense tensors."""
    D, H, ql = 80, 3, (200, 131)
    n = sum(ql)
    qkv = normal(38, n, 3, H, D, dtype=BF)
    do = normal(39, n, H, D, dtype=BF)
    att = vp.Attention(H, H, D)
    dense = run_attention(att, *(qkv[:, i].contiguous() for i in range(3)), do, cu(ql), cu(ql))
    packed = run_attention(att, qkv[:, 0], qkv[:, 1], qkv[:, 2], do, cu(ql), cu(ql))
    assert all(torch.equal(dense[x], packed[x]) for x in dense)
    outer = [qkv[:, i].transpose(0, 1).contiguous().transpose(0, 1) for i in range(3)]
    heads = run_attention(att, *outer, do.transpose(0, 1).contiguous().transpose(0, 1), cu(ql), cu(ql))
    assert all(torch.equal(dense[x], heads[x]) for x in dense)
    grad = torch.full_like(qkv, 7.0)
    att.backward(do, qkv[:, 0], qkv[:, 1], qkv[:, 2], dense["out"], dense["lse"], cu(ql), dq=grad[:, 0], dk=grad[:, 1],
                 dv=grad[:, 2])
    assert all(torch.equal(grad[:, i], dense[x]) for i, x in enumerate(("dq", "dk", "dv")))


def test_attention_neighbours_do_not_leak():
    """NaN and infinities in one sequence, and in the rows behind the last one,
    leave the others' results as they are; rows of no sequence are not written."""
    D, H, ql, tail = 72, 2, (130, 70, 61), 19
    n = sum(ql)
    t = {x: normal(40 + i, n + tail, H, D, dtype=BF) for i, x in enumerate(("q", "k", "v", "do"))}
    att = vp.Attention(H, H, D)
    c = cu(ql)

    def run(t):
        full = lambda: torch.full((n + tail, H, D), 3.0, dtype=BF, device=DEV)  # noqa: E731
        out, lse = att.forward(t["q"], t["k"], t["v"], c, out=full())
        grads = att.backward(t["do"], t["q"], t["k"], t["v"], out, lse, c, dq=full(), dk=full(), dv=full())
        return [out, *grads]
    clean = run(t)
    for x in t.values():
        x[130:165] = math.nan
        x[165:200] = math.inf
        x[n:] = math.nan
    dirty = run(t)
    for a, b in zip(clean, dirty):
        assert torch.equal(a[:130], b[:130]) and torch.equal(a[200:n], b[200:n])
        assert (a[n:] == 3.0).all() and (b[n:] == 3.0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_many_sequences(causal):
    """Thousands of short and empty sequences: each finds its rows (and the boundaries
    may begin and end inside the buffers)."""
    D, H = 64, 2
    g = torch.Generator().manual_seed(3)
    ql = torch.randint(0, 5, (3000,), generator=g).tolist()
    kl = [max(0, a + int(b)) for a, b in zip(ql, torch.randint(-1, 4, (3000,), generator=g))]
    nq, nk, pre = sum(ql), sum(kl), 7
    q, do = normal(100, pre + nq + 9, H, D, dtype=BF), normal(101, pre + nq + 9, H, D, dtype=BF)
    k, v = normal(102, nk, H, D, dtype=BF), normal(103, nk, H, D, dtype=BF)
    att = vp.Attention(H, H, D, causal=causal)
    out, lse = att.forward(q, k, v, cu(ql) + pre, cu(kl), out=torch.full_like(q, 2.0))
    dq, dk, dv = att.backward(do, q, k, v, out, lse, cu(ql) + pre, cu(kl), dq=torch.full_like(q, 2.0))
    mid = slice(pre, pre + nq)
    R, A = attention_ref(q[mid], k, v, ql, kl, causal, D ** -0.5, do[mid])
    check_attention({"out": out[mid], "lse": lse[:, mid], "dq": dq[mid], "dk": dk, "dv": dv}, R, A, nq, nk)
    for t in (out, dq):
        assert (t[:pre] == 2).all() and (t[pre + nq:] == 2).all()


@pytest.mark.parametrize("D,Hq,Hkv,ql,kl,causal", [
    (64, 16, 16, (64, 1, 130, 0, 63, 65, 200, 17, 128, 129, 5), None, False),
    (80, 16, 16, (64,) * 12, None, False),
    (72, 20, 20, (700, 12, 0, 128, 191, 1, 400), None, True),
    (96, 24, 12, (300, 129, 31, 3, 70), (64, 65, 0, 450, 1), False),
    (128, 24, 24, (40, 513, 64, 150), (30, 600, 64, 127), True),
    (128, 64, 16, tuple(range(1, 13)), tuple(range(150, 30, -10)), True),
    (8, 160, 160, (3, 0, 2), (66, 5, 300), False),
])
def test_attention_two_blocks_a_multiprocessor(D, Hq, Hkv, ql, kl, causal):
    """Short sequences in so many tiles that blocks of one tile share an SM; one sequence
    holds NaN, and the others' results do not."""
    kl = ql if kl is None else kl
    nq, nk = sum(ql), sum(kl)
    q, do = normal(110, nq, Hq, D, dtype=BF), normal(113, nq, Hq, D, dtype=BF)
    k, v = normal(111, nk, Hkv, D, dtype=BF), normal(112, nk, Hkv, D, dtype=BF)
    att = vp.Attention(Hq, Hkv, D, causal=causal)
    got = run_attention(att, q, k, v, do, cu(ql), cu(kl))
    R, A = attention_ref(q, k, v, ql, kl, causal, D ** -0.5, do)
    check_attention(got, R, A, nq, nk)
    a, b = sum(ql[:2]), sum(ql[:3])
    c, d = sum(kl[:2]), sum(kl[:3])
    for t, lo, hi in ((q, a, b), (do, a, b), (k, c, d), (v, c, d)):
        t[lo:hi] = math.nan
    dirty = run_attention(att, q, k, v, do, cu(ql), cu(kl))
    for n in ("out", "dq"):
        assert torch.equal(dirty[n][:a], got[n][:a]) and torch.equal(dirty[n][b:], got[n][b:]), n
    for n in ("dk", "dv"):
        assert torch.equal(dirty[n][:c], got[n][:c]) and torch.equal(dirty[n][d:], got[n][d:]), n
    assert torch.equal(dirty["lse"][:, :a], got["lse"][:, :a]) and torch.equal(dirty["lse"][:, b:], got["lse"][:, b:])


def test_attention_empty_sides():
    D, H = 64, 2
    some, none = normal(104, 5, H, D, dtype=BF), torch.empty(0, H, D, dtype=BF, device=DEV)
    att = vp.Attention(H, H, D)
    zero, five = torch.zeros(2, dtype=torch.int32, device=DEV), cu((5,))
    out, lse = att.forward(some, none, none, five, zero)               # no keys at all
    dq, dk, dv = att.backward(some, some, none, none, out, lse, five, zero)
    assert not out.any() and torch.isneginf(lse).all() and not dq.any() and dk.shape == dv.shape == (0, H, D)
    out, lse = att.forward(none, some, some, zero, five)               # no queries
    dq, dk, dv = att.backward(none, none, some, some, out, lse, zero, five)
    assert out.shape == dq.shape == (0, H, D) and not dk.any() and not dv.any()


def test_attention_divided_keys_leave_other_rows():
    """The joined form (one row on a long key axis) writes rows of sequences only."""
    D, H, n = 128, 2, 9000
    q, k, v = normal(47, 4, H, D, dtype=BF), normal(48, n + 50, H, D, dtype=BF), normal(49, n + 50, H, D, dtype=BF)
    k[n:] = v[n:] = math.nan
    att = vp.Attention(H, H, D)
    cq = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)      # rows 0 and 3 belong to nobody
    ck = torch.tensor([0, n, n], dtype=torch.int32, device=DEV)      # the second sequence has no keys
    assert B.pe_attention_workspace(att.h, 2, 4, n + 50, False) > 0
    out, lse = att.forward(q, k, v, cq, ck, out=torch.full_like(q, 5.0))
    R, A = attention_ref(q[1:2], k[:n], v[:n], (1,), (n,), False, D ** -0.5)
    close(out[1:2], R["out"], A["out"] + U[BF] * R["out"].abs(), "out")
    assert (out[0] == 5).all() and (out[3] == 5).all() and not out[2].any() and torch.isneginf(lse[:, 2]).all()


def test_attention_gradient_against_differences():
    """The inner product of each gradient with a direction against central
    differences of the 64-bit forward pass (h^2 error below 1e-7)."""
    D, H, ql, h = 64, 2, (50, 31), 1e-4
    n = sum(ql)
    x = [normal(50 + i, n, H, D, dtype=BF) for i in range(3)]
    do = normal(53, n, H, D, dtype=BF)
    got = run_attention(vp.Attention(H, H, D, causal=True), *x, do, cu(ql), cu(ql))
    R, A = attention_ref(*x, ql, ql, True, D ** -0.5, do)
    f = lambda a: (attention_ref(*a, ql, ql, True, D ** -0.5)[0]["out"] * do.double()).sum()  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        u = normal(54 + i, n, H, D).double()
        hi, lo = ([t.double() + (s * h * u if j == i else 0) for j, t in enumerate(x)] for s in (1, -1))
        num = float((f(hi) - f(lo)) / (2 * h))
        tol = float(((A[name] + U[BF] * R[name].abs()) * u.abs()).sum()) + 1e-6 * float((R[name] * u).abs().sum())
        assert abs(num - float((got[name].double() * u).sum())) <= tol, name


def test_attention_graph_replay_and_streams():
    """Captured calls replay on new data, and two graphs and an eager call on
    streams of their own give the same bits as one after the other."""
    D, H, ql = 80, 2, (257, 100)
    n = sum(ql)
    att = vp.Attention(H, H, D)
    c = cu(ql)
    sets = [[normal(60 + 10 * s + i, n, H, D, dtype=BF) for i in range(4)] for s in range(3)]
    want = [run_attention(att, *s[:3], s[3], c, c) for s in sets]
    static = [[torch.zeros_like(t) for t in sets[0]] for _ in range(2)]
    graphs, outs = [], []
    for st in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_attention(att, *st[:3], st[3], c, c))
        graphs.append(g)
    for a, b in ((0, 1), (1, 2)):
        for st, s in zip(static, (a, b)):
            for d, t in zip(st, sets[s]):
                d.copy_(t)
        torch.cuda.synchronize()
        s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        with torch.cuda.stream(s3):
            eager = run_attention(att, *sets[0][:3], sets[0][3], c, c)
        torch.cuda.synchronize()
        for got, s in ((outs[0], a), (outs[1], b), (eager, 0)):
            assert all(torch.equal(got[x], want[s][x]) for x in got)


def test_explicit_stream_argument():
    st = torch.cuda.Stream()
    x = normal(70, 64, 2, 64, dtype=BF)
    att = vp.Attention(2, 2, 64)
    torch.cuda.synchronize()
    out, _ = att.forward(x, x, x, cu((64,)), stream=st)
    y = vp.layer_norm(x, stream=st.cuda_stream)
    r, _ = vp.rope(x, None, torch.ones(1, 64, dtype=torch.int32, device=DEV), (32,), stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, att.forward(x, x, x, cu((64,)))[0]) and torch.equal(y, vp.layer_norm(x))
    assert torch.equal(r, vp.rope(x, None, torch.ones(1, 64, dtype=torch.int32, device=DEV), (32,))[0])


def test_attention_boundaries_out_of_contract_stay_inside():
    """Boundaries beyond the buffers or going back are held inside them: finite
    results for the good sequences, nothing else promised."""
    D, H, n = 64, 1, 300
    q, do = normal(80, n, H, D, dtype=BF), normal(81, n, H, D, dtype=BF)
    att = vp.Attention(H, H, D)
    c = torch.tensor([-5, 100, 60, 5000], dtype=torch.int32, device=DEV)
    out, lse = att.forward(q, q, q, c, out=torch.zeros_like(q))
    att.backward(do, q, q, q, out, lse, c)
    torch.cuda.synchronize()
    R, A = attention_ref(q[:60], q[:60], q[:60], (60,), (60,), False, D ** -0.5)
    assert att.last_error() == 0 and out.isfinite().all()


# ------------------------------------------------------------------ together


def test_tower_block_forward_and_backward():
    """Norm, projection, rotary positions and attention as a block uses them on two
    images and a clip, and back, against the same chain in 64 bits under autograd.
    Every stored bf16 tensor on the way is rounded once (U of its value); in the
    norm of a whole tensor the chain's ten or so roundings stay within 10 U."""
    grids, H, D = [(1, 10, 18), (2, 8, 6), (1, 16, 4)], 4, 72
    E = H * D
    pos, c = vp.vision_positions(grids, 2)
    n = pos.shape[1]
    x, wqkv = normal(90, n, E, dtype=BF), normal(91, 3 * E, E, dtype=BF, std=E ** -0.5)
    gamma, beta = normal(92, E, dtype=BF, std=0.1, mean=1.0), normal(93, E, dtype=BF, std=0.1)
    dout = normal(94, n, H, D, dtype=BF)
    sec = (D // 4, D // 4)
    att = vp.Attention(H, H, D)

    y, mean, rstd = vp.layer_norm(x, gamma, beta, 1e-6, stats=True)
    qkv = (y @ wqkv.t()).view(n, 3, H, D)
    q, k, v = qkv.unbind(1)
    vp.rope(q, k, pos[1:], sec, axial=True, out_q=q, out_k=k)
    out, lse = att.forward(q, k, v, c)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv.unbind(1)
    att.backward(dout, q, k, v, out, lse, c, dq=dq, dk=dk, dv=dv)
    vp.rope(dq, dk, pos[1:], sec, axial=True, inverse=True, out_q=dq, out_k=dk)
    dx, dgamma, dbeta = vp.layer_norm_backward((dqkv.view(n, 3 * E) @ wqkv).contiguous(), x, gamma, mean, rstd)

    xs, gs, bs = (t.double().requires_grad_() for t in (x, gamma, beta))
    ry = torch.nn.functional.layer_norm(xs, (E,), gs, bs, 1e-6)
    rq, rk, rv = (ry @ wqkv.double().t()).view(n, 3, H, D).unbind(1)
    rq, rk = (rope_ref(t, pos[1:], sec, 1e4, True, 1.0) for t in (rq, rk))
    b = c.tolist()
    parts = []
    for lo, hi in zip(b, b[1:]):
        s = torch.einsum("ihd,jhd->hij", rq[lo:hi], rk[lo:hi]) * D ** -0.5
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), rv[lo:hi]))
    ro = torch.cat(parts)
    ro.backward(dout.double())
    for got, ref, name in ((out, ro, "out"), (dx, xs.grad, "dx"), (dgamma, gs.grad, "dgamma"), (dbeta, bs.grad, "dbeta")):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= 10 * U[BF], (name, rel)


# ------------------------------------------------------------------ refusals on the device


def test_attention_refuses():
    x = normal(95, 64, 2, 64, dtype=BF)
    c = cu((64,))
    att = vp.Attention(2, 2, 64)
    with pytest.raises(TypeError):
        att.forward(x.float(), x, x, c)
    with pytest.raises(ValueError):
        att.forward(x[:, :1], x, x, c)
    with pytest.raises(TypeError):
        att.forward(x, x, x, c.long())
    with pytest.raises(ValueError):
        att.forward(x, x, x, c.cpu())
    with pytest.raises(ValueError):
        att.forward(x, x, x, c, cu((32, 32)))
    with pytest.raises(PEError) as e:                               # strides that no 16-byte access can follow
        att.forward(normal(96, 64, 2, 66, dtype=BF)[..., :64], x, x, c)
    assert e.value.status == "PE_ERR_ALIGN"
    with pytest.raises(PEError) as e:
        att.forward(x.flatten()[:64].expand(64, 2, 64), x, x, c)     # overlapping rows
    assert e.value.status == "PE_ERR_SHAPE"
    with pytest.raises(PEError) as e:                               # an output whose heads overlap
        att.forward(x, x, x, c, out=torch.empty(64 * 128 + 64, dtype=BF, device=DEV).as_strided((64, 2, 64), (64, 64, 1)))
    assert e.value.status == "PE_ERR_SHAPE"
    for bad in ((3, 2, 64, 0.1), (2, 2, 12, 0.1), (2, 2, 64, 0.0), (2, 2, 64, math.inf), (0, 1, 64, 0.1)):
        with pytest.raises(PEError) as e:
            B.pe_attention_create(*bad, False)
        assert e.value.status == "PE_ERR_INVALID_ARG"
    with pytest.raises(PEError) as e:
        vp.Attention(1, 1, 136)
    assert e.value.status == "PE_ERR_UNSUPPORTED"
    out, lse = att.forward(x, x, x, c)
    with pytest.raises(PEError) as e:                               # a workspace that is too small
        B.pe_attention_backward(att.h, 1, c.data_ptr(), 64, c.data_ptr(), 64, *[B.pe_heads(x.data_ptr(), 128, 64)] * 4,
                                lse.data_ptr(), *[B.pe_heads(x.data_ptr(), 128, 64)] * 4, lse.data_ptr(), 16, 0)
    assert e.value.status == "PE_ERR_SHAPE"


def test_layer_norm_workspace_is_checked():
    x = normal(97, 64, 64)
    _, mean, rstd = vp.layer_norm(x, stats=True)
    g = torch.empty(64, device=DEV)
    with pytest.raises(PEError) as e:
        B.pe_layernorm_backward(x.data_ptr(), x.data_ptr(), 0, 64, 64, None, 0, mean.data_ptr(), rstd.data_ptr(),
                                x.data_ptr(), g.data_ptr(), g.data_ptr(), g.data_ptr(), 16, 0)
    assert e.value.status == "PE_ERR_SHAPE"
