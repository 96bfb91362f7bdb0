"""Host side of the weight gradient: the division of its tiles among
workgroups (the library's own header, walked on the CPU) and the refusals of
its C entry."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000                        # a pointer that is never followed: every call below is refused first
OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 5


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def test_every_division_covers_each_tile_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "levels")
    subprocess.run([cxx, "-O2", "-std=c++17", "-D__host__=", "-D__device__=",
                    "-I" + os.path.join(ROOT, "fac_whitening_amd", "csrc"),
                    os.path.join(ROOT, "tests", "wgrad_levels_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout


def _call(fw, **change):
    ck = fw.ActCkpt(P, 1024, P, fw.E4M3)
    a = dict(delta=P, dtype=fw.BF16, ldd=64, m=64, ck=ck, T=500, d=1000, alpha=1.0, acc=0, W=P, ldw=1000, work=P,
             bytes=None, stream=None)
    a.update(change)
    if a["bytes"] is None:
        a["bytes"] = fw._lib.gift_weight_grad_workspace_bytes(a["T"], a["m"], a["d"], a["dtype"])
    return fw._lib.gift_weight_grad(*a.values())


def test_refusals(fw):
    for change in (dict(work=None), dict(work=P + 8), dict(W=P + 2), dict(ldw=999), dict(ldd=63), dict(m=0), dict(T=-1),
                   dict(dtype=7), dict(delta=P + 1)):
        assert _call(fw, bytes=1 << 40, **change) == INVALID, change
    for dt in (fw.BF16, fw.FP16, fw.FP32):
        need = fw._lib.gift_weight_grad_workspace_bytes(500, 64, 1000, dt)
        assert need > 0
        assert _call(fw, dtype=dt, bytes=need - 1) == WORKSPACE
    big = 1 << 24
    assert _call(fw, m=big, d=big, ldd=big, ldw=big, ck=fw.ActCkpt(P, big, P, fw.E4M3), bytes=1 << 60) == UNSUPPORTED


def test_workspace_is_bounded(fw):
    """Pieces of split tiles: never more than 512 + 512 tiles of 128 x 128 or
    256 + 256 of 256 x 256, whatever the sizes."""
    f = fw._lib.gift_weight_grad_workspace_bytes
    for dt in (fw.BF16, fw.FP16, fw.FP32):
        for T in (1, 63, 64, 1000, 16384, 1 << 20, 1 << 39):
            for m, d in ((1, 1), (8, 8), (64, 256), (1001, 2731), (1536, 6144), (4096, 16384), (1 << 24, 1 << 24)):
                # levels of a division: the pieces of each are at most its workgroups, and each level leaves
                # at most half of what its workgroups had, so the sum stays below 2 (workgroups + tiles)
                assert 0 < f(T, m, d, dt) <= 2 * (256 + 256) * 256 * 256 * 4 + 512, (T, m, d, dt)
    assert f(-1, 8, 8, fw.BF16) == 0 and f(1, 8, 8, 9) == 0 and f(1, 1 << 25, 8, fw.BF16) == 0
