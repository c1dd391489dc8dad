"""How the tensor-memory attention kernel leaves when one of its bounded waits has run out, on the CPU: the code
that orders it is compiled for the host, with threads for warps and CTAs."""
from __future__ import annotations

import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent


def _run(tmp_path, name, *args):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / name
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-pthread", "-I", str(ROOT / "layer_wise_paged_gb300" / "csrc"),
                        str(ROOT / "tests" / "host" / f"{name}.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_no_warp_is_left_waiting(tmp_path):
    """Whichever wait runs out, and whenever, every softmax warp comes to the end of its steps."""
    assert "meet: ok" in _run(tmp_path, "attend_meet")


def test_counters_are_zero_after_shares_that_gave_up(tmp_path):
    """A job's parts are joined once if all came, never otherwise, and its counter is cleared either way."""
    assert "shares: ok" in _run(tmp_path, "attend_shares")
