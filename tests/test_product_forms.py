"""Which form of its kernels a call of the gated block or of the weight
gradient takes (the library's own header, compiled for the host), and that the
division of a product's tiles that a kernel asks for piece by piece is the one
that the host counts."""
import os
import shutil
import subprocess

import pytest

from product_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _compile(tmp_path, name):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / name)
    subprocess.run([cxx, "-O2", "-std=c++17", "-D__host__=", "-D__device__=",
                    "-I" + os.path.join(ROOT, "fac_whitening_amd", "csrc"),
                    os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe], check=True)
    return exe


def test_every_form_has_its_sizes(tmp_path):
    """The sizes that the GPU tests run take the forms they are listed for, every form among them."""
    ask = "".join(f"{op} {t} {T} {d} {f}\n" for op, t, (T, d, f), _ in FORMS)
    out = subprocess.run([_compile(tmp_path, "product_plan_check")], input=ask, capture_output=True, text=True, check=True)
    got = out.stdout.splitlines()
    assert len(got) == len(FORMS)
    wrong = [(f, g) for f, g in zip(FORMS, got) if f[3] != g]
    assert not wrong, wrong
    # both tile sizes, whole and split, of every product and type
    have = {(op, t, form) for op, t, _, form in FORMS}
    for op in ("forward", "dx", "wgrad"):
        for t in ("16", "fp32"):
            for side in ("128", "256"):
                mine = {form for o, u, form in have if (o, u) == (op, t) and form.startswith(side)}
                assert any(form.endswith("none") for form in mine), (op, t, side)
                assert any(not form.endswith("none") for form in mine), (op, t, side)


def test_pieces_one_at_a_time(tmp_path):
    out = subprocess.run([_compile(tmp_path, "product_pieces_check")], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout
