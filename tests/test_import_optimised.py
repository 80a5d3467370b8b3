"""The package under every level of the interpreter's optimisation."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("flag", ["-O", "-OO"])  # (without assertions; without docstrings too)
def test_import(flag):
    pytest.importorskip("torch")
    code = "import fp32_gemm_major_amd as sg; print(sg.Mx8.nbytes(3, 65), sg.Mx4.nbytes(3, 65))"
    run = subprocess.run([sys.executable, flag, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr
    assert run.stdout.split() == ["297", "153"]
