"""Compile the HIP library ``libsgemm.so`` in place for gfx950.

    python -m fp32_gemm_major_amd.build

The library is plain HIP (no torch symbols); hipcc cross-compiles it on a
machine without a GPU.  The source files are compiled side by side and linked.  Packed FP32 arithmetic is switched off for every HIP
source (``-packed-fp32-ops``): the VALU kernel then uses one v_fma_f32 per
multiply-add.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libsgemm.so")
SOURCES = [os.path.join(CSRC, name) for name in ("sgemm.hip", "mx.hip", "ce.hip")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def command(source: str, output: str, extra=()) -> list:
    """The hipcc line that compiles one source file."""
    return [HIPCC, *FLAGS, *extra, "-c", "-o", output, source]


def link_command(objects, output: str = LIBRARY) -> list:
    return [HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", output, *objects]


def _run(cmd, verbose: bool) -> None:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(cmd) + "\n" + proc.stderr)
    if verbose and proc.stderr:
        sys.stderr.write(proc.stderr)


def build(output: str = LIBRARY, verbose: bool = False) -> str:
    tmp = output + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
            list(pool.map(lambda so: _run(command(*so), verbose), zip(SOURCES, objects)))
        _run(link_command(objects, tmp), verbose)
    os.replace(tmp, output)
    return output


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
