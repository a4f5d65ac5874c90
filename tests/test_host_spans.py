"""Batch metadata of the serving operators that is out of range, on the CPU: the functions that turn
lengths and row offsets into rows, table columns and visible keys, compiled for the host."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from fp8_quantized_linear_amd import build as B  # noqa: E402


def _hipcc():
    try:
        return B._hipcc()
    except RuntimeError:
        return None


@pytest.mark.skipif(_hipcc() is None, reason="hipcc missing")
def test_spans_stay_inside_their_arrays(tmp_path):
    exe = str(tmp_path / "spans")
    src = os.path.join(ROOT, "tests", "host", "serving_spans.cpp")
    csrc = os.path.join(ROOT, "fp8_quantized_linear_amd", "csrc")
    flags = ["-std=c++17", "-O1", "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
             "-fno-sanitize-recover=all", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    r = subprocess.run([_hipcc(), *flags, "-I", csrc, "-I", os.path.join(ROOT, "include"), "-x", "hip", src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "cases" in r.stdout
