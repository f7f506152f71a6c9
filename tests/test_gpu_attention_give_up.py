"""Attention calls whose bounded waits run out, on the GPU: with a wait limit of
nanoseconds (the bounds-checking build takes one from PE_TEST_WAIT_NS) the kernels'
waits give up at once or part-way through.  Every block then ends with nothing in
flight, the handle reports PE_ERR_DEVICE_TIMEOUT, and the next call with the usual
limit gives the usual bits.  Nothing faults, traps or hangs."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from vlm_vision_patch_b200 import build

pytestmark = pytest.mark.gpu


def test_waits_that_run_out_are_reported_and_the_handle_stays_usable():
    lib = build.build(debug_bounds=True)
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "attention_give_up_cases.py")
    env = {k: v for k, v in os.environ.items() if k != "PE_TEST_WAIT_NS"}
    r = subprocess.run([sys.executable, child], env={**env, "PE_LIB": lib}, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    print(r.stdout)
    assert int(r.stdout.split()[0]) >= 20, r.stdout
