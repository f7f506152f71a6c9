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
