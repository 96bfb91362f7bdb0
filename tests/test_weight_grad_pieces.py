"""The numbers of the weight gradient's pieces, walked on the host with the
library's own header."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_place_of_the_workspace_has_a_piece(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "pieces")
    subprocess.run([cxx, "-O2", "-std=c++17", "-D__host__=", "-D__device__=",
                    "-I" + os.path.join(ROOT, "fac_whitening_amd", "csrc"),
                    os.path.join(ROOT, "tests", "wgrad_pieces_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout
