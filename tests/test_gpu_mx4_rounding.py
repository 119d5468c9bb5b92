"""The quantiser's corrected quotients against IEEE division, exhaustively: a program
of its own that includes the kernels' rounding header (tests/rounding/rounding.cu)."""
import os
import shutil
import subprocess

import pytest

from routed_expert_ffn_topk_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


def test_every_quotient(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "rounding", "rounding.cu")
    exe = str(tmp_path / "rounding")
    subprocess.run([nvcc, *build_mod.ARCH, "-O3", "-std=c++17", "-I" + build_mod.CSRC, src, "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout.split()
    assert out[0::3] == ["boundary", "silu"]
    assert int(out[1]) == 6 * 2 ** 23 * 8 * 13 and int(out[4]) == 2 ** 32 - 2 ** 24
    assert int(out[2]) == 0 and int(out[5]) == 0, out
