"""Timed cases of the vision-tower operators: rotary positions over several axes,
layer norm (forward, and backward with the weight's gradient) and attention over
packed sequences (forward, and backward by recomputing the probabilities).

`run` computes each operator in plain torch operations (32 bits inside, 64 for the
rotary angles) or, with `own` set, calls this repository's package.  Widths, head
counts and grids are those of the package's workloads (1280 and 1152 wide rows, 16
heads; the 16-image group; 64 frames of 64 x 64 patches) and, for the language side,
12 query heads on 2 key heads of 128 with rotary sections 16, 24, 24.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# the 16 images of the package's grouped workload, (t, h, w) in patches
IMAGES = ("1x72x68 1x92x52 1x92x48 1x42x22 1x70x68 1x90x84 1x10x18 1x60x54 1x76x78 1x40x72 1x64x86 1x22x18 "
          "1x36x36 1x66x46 1x76x56 1x66x78")


def grids_of(text):
    return [tuple(int(v) for v in g.split("x")) for g in text.split()]


def lens_of(text):
    """Sequence lengths: "5 7*3" is 5, 7, 7, 7."""
    parts = [(p.split("*") + ["1"])[:2] for p in text.split()]
    return [int(a) for a, n in parts for _ in range(int(n))]


def frame_lens(text):
    """One sequence for each frame of each item: the tower's attention stays inside a frame."""
    return " ".join("%d*%d" % (h * w, t) for t, h, w in grids_of(text))


def listed():
    ln = {"op": "layer_norm", "eps": 1e-6}
    rg = {"op": "rope_grid", "merge": 2, "theta": 10000.0}
    at = {"op": "attention"}
    return [
        # the norm before the first block on one 224 x 896 image: a few microseconds, latency counts
        {**ln, "name": "norm of one image", "rows": 1024, "width": 1280, "dtype": "bf16", "train": False},
        # training on the long video
        {**ln, "name": "norm training, long video", "rows": 131072, "width": 1280, "dtype": "bf16", "train": True},
        # fp32 training on an odd number of rows of the 1152-wide tower
        {**ln, "name": "norm training, fp32, odd rows", "rows": 7841, "width": 1152, "dtype": "fp32", "train": True},
        # q and k of one image in a packed projection
        {**rg, "name": "rotary, one image", "grids": "1x16x64", "heads": 16, "dim": 80, "dtype": "bf16"},
        # q and k of the long video, 1152-wide tower (16 heads of 72)
        {**rg, "name": "rotary, long video", "grids": "32x64x64", "heads": 16, "dim": 72, "dtype": "bf16"},
        # the language side's three-axis positions far into a long document, gradient direction, fp32
        {"op": "rope_text", "name": "rotary gradient, far text, fp32", "rows": 16387, "heads": 12, "kv": 2, "dim": 128,
         "sections": "16 24 24", "theta": 1e6, "far": 1000000, "dtype": "fp32"},
        # one image through one block's attention
        {**at, "name": "attention, one image", "q": "1024", "k": "", "heads": 16, "kv": 16, "dim": 80,
         "causal": False, "train": False},
        # the 16-image group, ragged
        {**at, "name": "attention, 16 images", "q": frame_lens(IMAGES), "k": "", "heads": 16, "kv": 16, "dim": 80,
         "causal": False, "train": False},
        # ... and its training step
        {**at, "name": "attention training, 16 images", "q": frame_lens(IMAGES), "k": "", "heads": 16, "kv": 16,
         "dim": 80, "causal": False, "train": True},
        # an 8-frame clip of the 1152-wide tower: four short sequences, lengths that end inside a tile
        {**at, "name": "attention training, short clip", "q": "196*4", "k": "", "heads": 16, "kv": 16, "dim": 72,
         "causal": False, "train": True},
        # the language side: causal, shared key heads, documents of different lengths
        {**at, "name": "causal training, shared heads", "q": "4096 1000 2048 1 517", "k": "", "heads": 12, "kv": 2,
         "dim": 128, "causal": True, "train": True},
        # one new token for each of 8 conversations over its keys and values
        {**at, "name": "attention, single tokens", "q": "1*8", "k": "16384 9000 4097 1 12288 777 8192 15000",
         "heads": 12, "kv": 2, "dim": 128, "causal": True, "train": False},
    ]


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "rope_grid", "rope_text", "attention", "attention", "attention"])
    if op == "layer_norm":
        width = 8 * log_between(rng, 8, 1024)
        rows = min(log_between(rng, 1, 131072), 131072 * 1280 // width)
        return {"op": op, "rows": rows, "width": width, "eps": rng.choice([1e-6, 1e-5]),
                "dtype": rng.choice(["bf16", "fp32"]), "train": rng.random() < 0.6}
    if op == "rope_grid":
        merge = rng.choice([1, 2, 2, 3])
        items = []
        left = 65536
        for _ in range(log_between(rng, 1, 40)):
            t, h, w = log_between(rng, 1, 8), merge * log_between(rng, 2, 36), merge * log_between(rng, 2, 36)
            if t * h * w <= left:
                items.append("%dx%dx%d" % (t, h, w))
                left -= t * h * w
        return {"op": op, "grids": " ".join(items), "merge": merge, "theta": 10000.0, "heads": rng.choice([4, 12, 16]),
                "dim": rng.choice([64, 72, 80, 128]), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "rope_text":
        sections, dim = rng.choice([("16 24 24", 128), ("8 12 12", 64), ("12 10 10", 96), ("64", 128)])
        return {"op": op, "rows": log_between(rng, 1, 32768), "heads": rng.choice([8, 12, 28]), "kv": rng.choice([1, 2, 4]),
                "dim": dim, "sections": sections, "theta": rng.choice([1e4, 1e6]), "far": log_between(rng, 1000, 1000000),
                "dtype": rng.choice(["bf16", "fp32"])}
    kv = rng.choice([1, 2, 4, 16])
    heads = kv * rng.choice([1, 1, 2, 6]) if kv < 16 else 16
    causal = rng.random() < 0.35
    own_keys = rng.random() < 0.25                      # keys of their own: a cache before the new rows
    q, k, pairs = [], [], 200_000_000 // heads * 8
    for _ in range(log_between(rng, 1, 24)):
        a = log_between(rng, 1, 6000)
        b = a
        if own_keys:
            a = rng.choice([1, 1, log_between(rng, 1, 300)])
            b = log_between(rng, 1, 12000) + (a if causal else 0)
        if a * b <= pairs:
            q.append(str(a))
            k.append(str(b))
            pairs -= a * b
    return {"op": op, "q": " ".join(q), "k": " ".join(k) if own_keys else "", "heads": heads, "kv": kv,
            "dim": rng.choice([64, 72, 80, 96, 128]), "causal": causal, "train": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "layer_norm":
        dt, n, e = DTYPES[case["dtype"]], case["rows"], case["width"]
        s["x"] = normal(n, e, dtype=dt, std=1.5, mean=0.3)
        s["gamma"], s["beta"] = normal(e, dtype=dt, std=0.1, mean=1.0), normal(e, dtype=dt, std=0.1)
        if case["train"]:
            s["dy"] = normal(n, e, dtype=dt)
        return s
    if op == "rope_grid":
        s["grids"] = grids_of(case["grids"])
        n = sum(t * h * w for t, h, w in s["grids"])
        qkv = normal(n, 3, case["heads"], case["dim"], dtype=DTYPES[case["dtype"]])   # the packed projection
        s["q"], s["k"] = qkv[:, 0], qkv[:, 1]
        s["sections"] = (case["dim"] // 4, case["dim"] // 4)                           # height, width
        return s
    if op == "rope_text":
        n, dt = case["rows"], DTYPES[case["dtype"]]
        s["q"], s["k"] = normal(n, case["heads"], case["dim"], dtype=dt), normal(n, case["kv"], case["dim"], dtype=dt)
        s["sections"] = tuple(int(v) for v in case["sections"].split())
        s["pos"] = torch.randint(0, case["far"], (len(s["sections"]), n), generator=g, device=DEV, dtype=torch.int32)
        return s
    hq, hk, d, dt = case["heads"], case["kv"], case["dim"], torch.bfloat16
    s["q_lens"] = lens_of(case["q"])
    s["k_lens"] = lens_of(case["k"]) if case["k"] else s["q_lens"]
    nq, nk = sum(s["q_lens"]), sum(s["k_lens"])
    if hq == hk and not case["k"]:
        qkv = normal(nq, 3, hq, d, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, 0], qkv[:, 1], qkv[:, 2]
    else:
        s["q"], s["k"], s["v"] = normal(nq, hq, d, dtype=dt), normal(nk, hk, d, dtype=dt), normal(nk, hk, d, dtype=dt)

    def cu(lens):
        return torch.tensor([0] + lens).cumsum(0).to(device=DEV, dtype=torch.int32)

    s["cu_q"] = cu(s["q_lens"])
    s["cu_k"] = cu(s["k_lens"]) if case["k"] else s["cu_q"]
    if case["train"]:
        s["do"] = normal(nq, hq, d, dtype=dt)
    if own:
        import vlm_vision_patch_b200 as vp
        s["attention"] = vp.Attention(hq, hk, d, causal=case["causal"])
    return s


# ------------------------------------------------------------------ the operators


def run(s):
    return (own_run if own else plain_run)(s)


def own_run(s):
    import vlm_vision_patch_b200 as vp
    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        if not case["train"]:
            return {"y": vp.layer_norm(s["x"], s["gamma"], s["beta"], case["eps"])}
        y, mean, rstd = vp.layer_norm(s["x"], s["gamma"], s["beta"], case["eps"], stats=True)
        dx, dgamma, dbeta = vp.layer_norm_backward(s["dy"], s["x"], s["gamma"], mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "rope_grid":
        pos, cu = vp.vision_positions(s["grids"], case["merge"])
        q, k = vp.rope(s["q"], s["k"], pos[1:], s["sections"], theta=case["theta"], axial=True)
        return {"q": q, "k": k, "pos": pos, "cu": cu}
    if op == "rope_text":
        q, k = vp.rope(s["q"], s["k"], s["pos"], s["sections"], theta=case["theta"], inverse=True)
        return {"dq": q, "dk": k}
    att = s["attention"]
    out, lse = att.forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    if not case["train"]:
        return {"out": out, "lse": lse}
    dq, dk, dv = att.backward(s["do"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def plain_run(s):
    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        return plain_norm(s, case)
    if op == "rope_grid":
        pos, cu = plain_positions(s["grids"], case["merge"])
        sec = torch.tensor(s["sections"], device=DEV)
        step = torch.cat([torch.arange(n, device=DEV, dtype=torch.float64) / n for n in s["sections"]])
        q, k = plain_rotate(s["q"], s["k"], pos[1:], sec, step, case["theta"], 1.0)
        return {"q": q, "k": k, "pos": pos, "cu": cu}
    if op == "rope_text":
        sec = torch.tensor(s["sections"], device=DEV)
        step = torch.arange(sum(s["sections"]), device=DEV, dtype=torch.float64) / sum(s["sections"])
        q, k = plain_rotate(s["q"], s["k"], s["pos"], sec, step, case["theta"], -1.0)
        return {"dq": q, "dk": k}
    return plain_attention(s, case)


def plain_norm(s, case):
    x, gamma, beta = s["x"].float(), s["gamma"].float(), s["beta"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt(c.square().mean(1, keepdim=True) + case["eps"])
    xh = c * rstd
    y = (xh * gamma + beta).to(s["x"].dtype)
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].float()
    a = dy * gamma
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    dt = s["gamma"].dtype
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx.to(s["x"].dtype),
            "dgamma": (dy * xh).sum(0, dtype=torch.float64).to(dt), "dbeta": dy.sum(0, dtype=torch.float64).to(dt)}


def plain_positions(grids, m):
    """Rows in merge order: frames one behind the other, m x m windows row by row inside a frame."""
    g = torch.tensor(grids, device=DEV)
    frames = g[:, 1:].repeat_interleave(g[:, 0], 0)                      # (h, w) of each frame
    t = torch.cat([torch.arange(int(v[0]), device=DEV) for v in grids])
    sizes = frames[:, 0] * frames[:, 1]
    cu = torch.nn.functional.pad(sizes.cumsum(0), (1, 0))
    frame = torch.arange(len(frames), device=DEV).repeat_interleave(sizes)
    r = torch.arange(len(frame), device=DEV) - cu[frame]
    across = frames[frame, 1] // m
    win, at = r // (m * m), r % (m * m)
    pos = torch.stack([t[frame], win // across * m + at // m, win % across * m + at % m])
    return pos.int(), cu.int()


def plain_rotate(q, k, pos, sections, step, theta, sign):
    axis = torch.arange(len(sections), device=DEV).repeat_interleave(sections)
    angle = pos.double()[axis].t() * theta ** -step * sign               # [N, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    n = cos.shape[-1]

    def turn(x):
        a, b = x[..., :n].float(), x[..., n:2 * n].float()
        return torch.cat([(a * cos - b * sin).to(x.dtype), (b * cos + a * sin).to(x.dtype), x[..., 2 * n:]], -1)

    return turn(q), turn(k)


def plain_attention(s, case):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    share, scale = hq // hk, d ** -0.5
    out, lse = torch.zeros_like(q, memory_format=torch.contiguous_format), q.new_empty(hq, len(q))
    grads = None
    if case["train"]:
        do = s["do"].float()
        grads = [torch.zeros_like(t, memory_format=torch.contiguous_format) for t in (q, k, v)]
    a = b = 0
    for m, n in zip(s["q_lens"], s["k_lens"]):                           # one sequence: all its heads at once
        rows, cols = slice(a, a + m), slice(b, b + n)
        a, b = a + m, b + n
        qs = q[rows].transpose(0, 1)                                     # [hq, m, d]
        ks, vs = (t[cols].transpose(0, 1).repeat_interleave(share, 0) for t in (k, v))
        p = qs @ ks.transpose(1, 2) * scale
        if case["causal"]:
            p.masked_fill_(torch.arange(n, device=DEV) > torch.arange(m, device=DEV)[:, None] + (n - m), -math.inf)
        top = p.amax(-1, keepdim=True)
        total = (p - top).exp().sum(-1, keepdim=True)
        lse[:, rows] = (top + total.log())[..., 0]
        p = p.sub_(top).exp_().div_(total)
        o = p @ vs
        out[rows] = o.transpose(0, 1)
        if grads is None:
            continue
        dos = do[rows].transpose(0, 1)
        dv = p.transpose(1, 2) @ dos
        ds = p * (dos @ vs.transpose(1, 2) - (dos * o).sum(-1, keepdim=True)) * scale
        grads[0][rows] = (ds @ ks).transpose(0, 1)
        grads[1][cols] = (ds.transpose(1, 2) @ qs).unflatten(0, (hk, share)).sum(1).transpose(0, 1)
        grads[2][cols] = dv.unflatten(0, (hk, share)).sum(1).transpose(0, 1)
    dt = s["q"].dtype
    if grads is None:
        return {"out": out.to(dt), "lse": lse}
    return {"out": out.to(dt), "lse": lse, "dq": grads[0].to(dt), "dk": grads[1].to(dt), "dv": grads[2].to(dt)}


# ------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "layer_norm":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["width"]
        # forward: x in, y out; training: x and dy in, y and dx out (x is read once for both), statistics out
        if not case["train"]:
            return {"bytes": size * (2 * n + 2 * case["width"]), "flops": 8 * n}
        return {"bytes": size * (4 * n + 4 * case["width"]) + 8 * case["rows"], "flops": 20 * n}
    if op in ("rope_grid", "rope_text"):
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "rope_grid":
            rows, heads, axes = sum(t * h * w for t, h, w in grids_of(case["grids"])), 2 * case["heads"], 3
        else:
            rows, heads, axes = case["rows"], case["heads"] + case["kv"], len(case["sections"].split())
        return {"bytes": 2 * size * rows * heads * case["dim"] + 4 * axes * rows, "flops": 3 * rows * heads * case["dim"]}
    ql = lens_of(case["q"])
    kl = lens_of(case["k"]) if case["k"] else ql
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    if case["causal"]:   # the sum over rows i of how many keys j <= i + n - m there are
        pairs = sum(sum(max(0, i + n - m + 1) for i in range(m)) for m, n in zip(ql, kl))
    else:
        pairs = sum(m * n for m, n in zip(ql, kl))
    nq, nk = sum(ql), sum(kl)
    size = 2 * d * (2 * nq * hq + 2 * nk * hk) + 4 * nq * hq             # q, out, k, v and lse
    if case["train"]:
        size += 2 * d * (2 * nq * hq + 2 * nk * hk)                      # do, dq, dk, dv
    return {"bytes": size, "flops": (14 if case["train"] else 4) * pairs * hq * d}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "layer_norm":
        return exact_norm(s, case)
    if op == "rope_grid":
        return exact_grid(s, case)
    if op == "rope_text":
        n = sum(s["sections"])
        rates = [(a, case["theta"] ** (-i / n)) for i, a in enumerate(a for a, m in enumerate(s["sections"]) for _ in range(m))]
        return {"dq": exact_turn(s["q"], s["pos"], rates, True), "dk": exact_turn(s["k"], s["pos"], rates, True)}
    return exact_attention(s, case)


def exact_norm(s, case):
    x, w = s["x"].double(), s["gamma"].double()
    n = x.shape[1]
    mean = x.sum(1) / n
    var = ((x * x).sum(1) - n * mean * mean) / n
    rstd = (var + case["eps"]) ** -0.5
    z = (x - mean[:, None]) * rstd[:, None]
    y = z * w + s["beta"].double()
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].double()
    # the Jacobian of z applied to dy * w: (I - (1 1^T + z z^T) / n) * rstd
    t = dy * w
    dx = (t - (t.sum(1, keepdim=True) + z * torch.einsum("ij,ij->i", t, z)[:, None]) / n) * rstd[:, None]
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, z), "dbeta": dy.sum(0)}


def exact_turn(x, pos, rates, back):
    """Each pair as a complex number, turned by e^(i angle); what is behind the pairs stays."""
    n = len(rates)
    angle = torch.stack([pos[a].double() * r for a, r in rates], 1)
    z = torch.complex(x[..., :n].double(), x[..., n:2 * n].double())
    z = z * torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
    return torch.cat([z.real, z.imag, x[..., 2 * n:].double()], -1)


def exact_grid(s, case):
    m, rows, sizes = case["merge"], [], [0]
    for t, h, w in s["grids"]:
        row = torch.arange(h, device=DEV)[:, None].expand(h, w)
        col = torch.arange(w, device=DEV)[None].expand(h, w)
        order = torch.stack([row, col]).reshape(2, h // m, m, w // m, m).permute(0, 1, 3, 2, 4).reshape(2, -1)
        for f in range(t):
            rows.append(torch.cat([torch.full_like(order[:1], f), order]))
            sizes.append(sizes[-1] + h * w)
    pos = torch.cat(rows, 1).int()
    rates = [(a, case["theta"] ** (-i / n)) for a, n in enumerate(s["sections"]) for i in range(n)]
    return {"q": exact_turn(s["q"], pos[1:], rates, False), "k": exact_turn(s["k"], pos[1:], rates, False),
            "pos": pos, "cu": torch.tensor(sizes, device=DEV, dtype=torch.int32)}


def exact_attention(s, case):
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    nq, nk = sum(s["q_lens"]), sum(s["k_lens"])
    if sum(m * n for m, n in zip(s["q_lens"], s["k_lens"])) * hq * d > 2e12:
        return None
    new = lambda *shape: torch.zeros(*shape, device=DEV, dtype=torch.float64)  # noqa: E731
    out, lse = new(nq, hq, d), new(hq, nq)
    dq, dk, dv = new(nq, hq, d), new(nk, hk, d), new(nk, hk, d)
    for h in range(hq):
        i = j = 0
        for m, n in zip(s["q_lens"], s["k_lens"]):
            q, k, v = s["q"][i:i + m, h].double(), s["k"][j:j + n, h * hk // hq].double(), s["v"][j:j + n, h * hk // hq].double()
            logits = torch.einsum("md,nd->mn", q, k) / math.sqrt(d)
            if case["causal"]:
                logits = logits + torch.full((m, n), -math.inf, device=DEV, dtype=torch.float64).triu(n - m + 1)
            lse[h, i:i + m] = torch.logsumexp(logits, 1)
            w = torch.exp(logits - lse[h, i:i + m, None])
            out[i:i + m, h] = torch.einsum("mn,nd->md", w, v)
            if case["train"]:
                do = s["do"][i:i + m, h].double()
                dv[j:j + n, h * hk // hq] += torch.einsum("mn,md->nd", w, do)
                dw = torch.einsum("md,nd->mn", do, v)
                dl = w * (dw - torch.einsum("mn,mn->m", w, dw)[:, None]) / math.sqrt(d)
                dq[i:i + m, h] = torch.einsum("mn,nd->md", dl, k)
                dk[j:j + n, h * hk // hq] += torch.einsum("mn,md->nd", dl, q)
            i, j = i + m, j + n
    if not case["train"]:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
