"""Child process of test_gpu_attention_give_up: runs attention calls whose waits run
out, with the library that PE_LIB names (the bounds-checking build, whose wait limit
PE_TEST_WAIT_NS sets), and prints how many of them were reported.

Not a test module (pytest collects test_*.py only)."""
from __future__ import annotations

import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import vlm_vision_patch_b200 as vp  # noqa: E402
from vlm_vision_patch_b200 import _binding as B  # noqa: E402

DEV, TIMEOUT = "cuda:0", 8
# D, Hq, Hkv, causal, query lengths, key lengths
SHAPES = [
    (80, 2, 2, False, (700,), (700,)),
    (128, 12, 2, True, (300, 517), (300, 517)),               # dk and dv in parts
    (64, 16, 16, False, (64,) * 12, (64,) * 12),              # blocks of one tile
    (128, 12, 2, True, (1, 2), (9000, 5120)),                 # the key axis divided
    (96, 2, 1, False, (40, 0, 200), (333, 7, 0)),
]
LIMITS = (0, 1, 5, 10, 20, 50, 200, 1000)                     # ns: at once, or part-way


def cu(lens):
    return torch.tensor([0, *lens]).cumsum(0).to(device=DEV, dtype=torch.int32)


def main() -> None:
    assert os.path.basename(B.LIB_PATH) == "libpe_debug.so", B.LIB_PATH
    reported = 0
    for D, Hq, Hkv, causal, ql, kl in SHAPES:
        g = torch.Generator(device=DEV).manual_seed(D + Hq)
        q, do = (torch.randn(sum(ql), Hq, D, generator=g, device=DEV).bfloat16() for _ in range(2))
        k, v = (torch.randn(sum(kl), Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
        att = vp.Attention(Hq, Hkv, D, causal=causal)
        cq, ck = cu(ql), cu(kl)

        def both():
            out, lse = att.forward(q, k, v, cq, ck)
            return [out, lse, *att.backward(do, q, k, v, out, lse, cq, ck)]
        want = both()
        torch.cuda.synchronize()
        assert att.last_error() == 0
        for limit in LIMITS:
            for backward in (False, True):
                os.environ["PE_TEST_WAIT_NS"] = str(limit)
                t0 = time.perf_counter()
                if backward:
                    att.backward(do, q, k, v, want[0], want[1], cq, ck)
                else:
                    att.forward(q, k, v, cq, ck)
                torch.cuda.synchronize()
                assert time.perf_counter() - t0 < 30
                del os.environ["PE_TEST_WAIT_NS"]
                status = att.last_error()
                assert status == TIMEOUT if limit == 0 else status in (0, TIMEOUT), (D, limit, backward, status)
                assert att.last_error() == 0                  # read and cleared
                reported += status == TIMEOUT
                assert all(torch.equal(a, b) for a, b in zip(both(), want)), (D, limit, backward)
                torch.cuda.synchronize()
                assert att.last_error() == 0
    print(f"{reported} of {2 * len(LIMITS) * len(SHAPES)} calls reported")


if __name__ == "__main__":
    main()
