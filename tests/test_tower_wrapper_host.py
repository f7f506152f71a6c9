"""What the vision-tower wrappers refuse before they look at a device (no GPU)."""
from __future__ import annotations

import pytest
import torch

import vlm_vision_patch_b200 as vp
from vlm_vision_patch_b200 import _binding as B


def test_recorded_calls_take_no_output_tensors():
    x, pos = torch.zeros(4, 2, 8), torch.zeros(1, 4, dtype=torch.int32)
    w = x.clone().requires_grad_()
    for call in (lambda: vp.rope(w, None, pos, (4,), out_q=x), lambda: vp.rope(x, w, pos, (4,), out_k=x),
                 lambda: vp.rope(x, None, pos, (4,), out_q=w), lambda: vp.layer_norm(w, out=x),
                 lambda: vp.layer_norm(x, w[0, 0], out=x), lambda: vp.layer_norm(x, out=w)):
        with pytest.raises(ValueError, match="output tensors"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()


def test_positions_are_not_put_on_the_host():
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ValueError, match="CUDA device"):
            vp.vision_positions([(1, 2, 2)], 2, device=device)


def test_rope_refuses_rates_that_are_not_finite():
    """theta^(-i/S) overflows for the least numbers above 0: position 0 would turn by 0 * inf."""
    def status(theta, sections, axial):
        q = B.pe_heads(4096, 512, 256)
        try:
            B.pe_rope(q, q, B.PE_F32, 0, 2, 2, 256, None, sections, theta, axial, False, q, q, 0)   # no rows: nothing is launched
        except vp.PEError as e:
            return e.status
        return "PE_OK"
    assert status(5e-324, (128,), False) == "PE_ERR_UNSUPPORTED" and status(5e-324, (64, 64), True) == "PE_ERR_UNSUPPORTED"
    assert status(1e-300, (128,), False) == "PE_OK" and status(1e300, (128,), False) == "PE_OK"
    assert status(5e-324, (2, 2), True) == "PE_OK"             # the fastest pair's rate is theta^(-1/2)
