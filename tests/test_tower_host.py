"""Refusals of the vision-tower calls (no GPU): every bad argument is answered
before anything is launched, with pointers that nothing reads."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import vlm_vision_patch_b200 as vp
from vlm_vision_patch_b200 import PEError
from vlm_vision_patch_b200 import _binding as B

P = 4096        # an aligned address that must not be touched
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vlm_vision_patch_b200 import build
    build.build()


def status(fn, *a):
    try:
        fn(*a)
    except PEError as e:
        return e.status
    return "PE_OK"


def h(ptr=P, row=64, head=8):
    return B.pe_heads(ptr, row, head)


ROPE = dict(q=h(), k=h(), dt=1, N=4, Hq=2, Hk=2, D=8, pos_ptr=P, sections=(4,), theta=1e4, axial=False, inverse=False,
            q_out=h(), k_out=h(), stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), "PE_ERR_INVALID_ARG"), (dict(Hq=0), "PE_ERR_INVALID_ARG"), (dict(D=0), "PE_ERR_INVALID_ARG"),
    (dict(theta=0.0), "PE_ERR_INVALID_ARG"), (dict(theta=math.inf), "PE_ERR_INVALID_ARG"),
    (dict(theta=math.nan), "PE_ERR_INVALID_ARG"), (dict(sections=()), "PE_ERR_INVALID_ARG"),
    (dict(sections=(-1, 5)), "PE_ERR_INVALID_ARG"), (dict(sections=(0,)), "PE_ERR_SHAPE"),
    (dict(sections=(5,)), "PE_ERR_SHAPE"), (dict(sections=(1,) * 5, D=64), "PE_ERR_UNSUPPORTED"),
    (dict(sections=(129,), D=512), "PE_ERR_UNSUPPORTED"), (dict(D=1025), "PE_ERR_UNSUPPORTED"),
    (dict(N=2 ** 31), "PE_ERR_UNSUPPORTED"), (dict(dt=2), "PE_ERR_DTYPE"), (dict(pos_ptr=None), "PE_ERR_INVALID_ARG"),
    (dict(pos_ptr=P + 2), "PE_ERR_ALIGN"), (dict(q=h(None)), "PE_ERR_INVALID_ARG"), (dict(k_out=h(None)), "PE_ERR_INVALID_ARG"),
    (dict(q=h(P + 1)), "PE_ERR_ALIGN"), (dict(dt=0, q_out=h(P + 2)), "PE_ERR_ALIGN"),
    (dict(q=h(P, -64)), "PE_ERR_INVALID_ARG"), (dict(q_out=h(P, 8, 8)), "PE_ERR_SHAPE"),
    (dict(k_out=h(P, 0, 8)), "PE_ERR_SHAPE"), (dict(k_out=h(P, 16, 4)), "PE_ERR_SHAPE"), (dict(N=0, pos_ptr=None, q=h(None)), "PE_OK"),
])
def test_rope_refuses(change, want):
    assert status(B.pe_rope, *{**ROPE, **change}.values()) == want


@pytest.mark.parametrize("grids,merge,want", [
    ([(1, 4, 4)], 0, "PE_ERR_INVALID_ARG"), ([(1, 4, 4)], 5, "PE_ERR_INVALID_ARG"), ([(1, 3, 4)], 2, "PE_ERR_SHAPE"),
    ([(1, 4, 6)], 4, "PE_ERR_SHAPE"), ([(0, 4, 4)], 2, "PE_ERR_SHAPE"), ([(1, -4, 4)], 2, "PE_ERR_SHAPE"),
    ([(2 ** 20, 2 ** 6, 2 ** 6)], 2, "PE_ERR_UNSUPPORTED"), ([(1, 2 ** 16, 2 ** 16)], 2, "PE_ERR_UNSUPPORTED"),
    ([(1, 2 ** 15, 2 ** 15), (1, 2 ** 15, 2 ** 15)], 2, "PE_ERR_UNSUPPORTED"),
])
def test_positions_refuse(grids, merge, want):
    assert status(B.pe_vision_positions, grids, merge, P, P, 0) == want


def test_positions_refuse_alignment_and_null():
    assert status(B.pe_vision_positions, [(1, 2, 2)], 2, P + 2, P, 0) == "PE_ERR_ALIGN"
    assert B.load().pe_vision_positions(1, None, 2, P, P, None) == 1
    assert B.load().pe_vision_positions(-1, None, 2, P, P, None) == 1
    with pytest.raises(ValueError):
        vp.vision_positions([(1, 2)], 2)
    with pytest.raises(ValueError):
        vp.vision_positions([(1, 0, 2)], 1)


FWD = dict(x=P, dt=1, N=4, E=64, gamma=P, beta=P, w_dt=1, eps=1e-6, y=P, mean=P, rstd=P, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), "PE_ERR_INVALID_ARG"), (dict(E=0), "PE_ERR_INVALID_ARG"), (dict(E=60), "PE_ERR_UNSUPPORTED"),
    (dict(E=16392), "PE_ERR_UNSUPPORTED"), (dict(N=2 ** 31), "PE_ERR_UNSUPPORTED"), (dict(dt=3), "PE_ERR_DTYPE"),
    (dict(w_dt=-1), "PE_ERR_DTYPE"), (dict(eps=-1.0), "PE_ERR_INVALID_ARG"), (dict(eps=math.nan), "PE_ERR_INVALID_ARG"),
    (dict(x=None), "PE_ERR_INVALID_ARG"), (dict(y=None), "PE_ERR_INVALID_ARG"), (dict(mean=None), "PE_ERR_INVALID_ARG"),
    (dict(x=P + 8), "PE_ERR_ALIGN"), (dict(gamma=P + 2), "PE_ERR_ALIGN"), (dict(mean=P + 2), "PE_ERR_ALIGN"),
    (dict(N=0, x=None, y=None), "PE_OK"),
])
def test_layer_norm_refuses(change, want):
    assert status(B.pe_layernorm_forward, *{**FWD, **change}.values()) == want


BWD = dict(dy=P, x=P, dt=1, N=4, E=64, gamma=P, w_dt=1, mean=P, rstd=P, dx=P, dgamma=P, dbeta=P, ws=P, n=1 << 20, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(dy=None), "PE_ERR_INVALID_ARG"), (dict(mean=None), "PE_ERR_INVALID_ARG"), (dict(dx=None), "PE_ERR_INVALID_ARG"),
    (dict(dgamma=None), "PE_ERR_INVALID_ARG"), (dict(E=12), "PE_ERR_UNSUPPORTED"), (dict(dt=9), "PE_ERR_DTYPE"),
    (dict(dbeta=P + 4), "PE_ERR_ALIGN"), (dict(ws=P + 4), "PE_ERR_ALIGN"), (dict(rstd=P + 1), "PE_ERR_ALIGN"),
])
def test_layer_norm_backward_refuses(change, want):
    assert status(B.pe_layernorm_backward, *{**BWD, **change}.values()) == want


def test_workspace_sizes_refuse():
    assert B.pe_layernorm_backward_workspace(-1, 64) == -1
    assert B.pe_layernorm_backward_workspace(4, 12) == -1
    assert B.pe_attention_workspace(None, 1, 4, 4, True) == -1


def test_attention_create_refuses_before_any_device_call():
    for bad in ((0, 1, 64, 0.1, 0), (2, 0, 64, 0.1, 0), (3, 2, 64, 0.1, 0), (2, 2, 4, 0.1, 0), (2, 2, 12, 0.1, 0),
                (2, 2, 64, 0.0, 0), (2, 2, 64, -1.0, 0), (2, 2, 64, math.nan, 0), (2, 2, 64, math.inf, 0), (2, 2, 64, 0.1, 2)):
        a = ctypes.c_void_p(1)
        assert B.load().pe_attention_create(*bad, ctypes.byref(a)) == 1 and not a.value
    a = ctypes.c_void_p(1)
    for bad in ((2, 2, 136, 0.1, 0), (2, 2, 64, 1e-21, 0), (2, 2, 64, 1e21, 0)):
        assert B.load().pe_attention_create(*bad, ctypes.byref(a)) == 7 and not a.value
    assert B.load().pe_attention_create(2, 2, 64, 0.1, 0, None) == 1
    assert B.pe_attention_last_error(None) == 1
    B.pe_attention_destroy(None)


def test_null_attention_handle():
    assert status(B.pe_attention_forward, None, 1, P, 4, P, 4, h(), h(), h(), h(), P, None, 0, 0) == "PE_ERR_INVALID_ARG"
    assert status(B.pe_attention_backward, None, 1, P, 4, P, 4, h(), h(), h(), h(), P, h(), h(), h(), h(), P, 64,
                  0) == "PE_ERR_INVALID_ARG"


def test_wrappers_want_device_tensors():
    x, pos = torch.zeros(4, 2, 8), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vp.rope(x, x, pos, (4,))
    with pytest.raises(ValueError, match="CUDA"):
        vp.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        vp.layer_norm_backward(x, x, None, x, x)
    a = vp.Attention.__new__(vp.Attention)
    a.heads = a.kv_heads = 2
    a.head_dim, a.h, a.dev = 8, None, 0
    c = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_q"):
        a.forward(x, x, x, c)
    with pytest.raises(ValueError, match="n_seq"):
        a.forward(x, x, x, c[None])
    with pytest.raises(ValueError, match="sequence counts"):
        a.forward(x, x, x, c, c[:1])
