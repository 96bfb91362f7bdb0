"""Sizes of the weight gradient whose tiles, counted in 32 bits, pass their
range: the workspace query and the call have to return, the call with a
refusal.  They run in a process of their own, so that one that does not return
ends as a failure (no GPU is needed: the pointers are never followed)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNSUPPORTED = 5

RUN = """
import sys
import fac_whitening_amd as fw
T, m, d, dt = map(int, sys.argv[1:])
P = 1 << 20
need = fw._lib.gift_weight_grad_workspace_bytes(T, m, d, dt)
status = fw._lib.gift_weight_grad(P, dt, m, m, fw.ActCkpt(P, (d + 31) // 32 * 32, P, fw.E4M3), T, d, 1.0, 0, P, d, P,
                                  1 << 50, None)
small = fw._lib.gift_weight_grad(P, dt, m, m, fw.ActCkpt(P, (d + 31) // 32 * 32, P, fw.E4M3), T, d, 1.0, 0, P, d, P,
                                 0, None)
print("done", need, status, small)
"""


@pytest.mark.parametrize("T,m,d,dt", [(1, 1 << 23, 1 << 22, 0), (64, 1 << 24, 1 << 21, 0), (64, 1 << 24, 1 << 23, 2),
                                      (64, 1 << 24, 12000000, 1), (64, 1 << 24, 1 << 22, 0), (1, 1 << 24, 1 << 24, 1)])
def test_outputs_beyond_a_launch(T, m, d, dt):
    out = subprocess.run([sys.executable, "-c", RUN, *map(str, (T, m, d, dt))], cwd=ROOT, capture_output=True,
                         text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    word, need, status, small = out.stdout.split()
    # no plan: no pieces of tiles to keep
    assert word == "done" and 0 < int(need) <= 512 and int(status) == UNSUPPORTED and int(small) == UNSUPPORTED
