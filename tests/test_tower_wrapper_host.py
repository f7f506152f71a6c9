"""What the vision-tower wrappers refuse before they look at a device (no GPU)."""
from __future__ import annotations

import pytest
import torch

import vlm_vision_patch_b200 as vp


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
