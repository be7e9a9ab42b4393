"""Numbers that a launcher asks the driver for belong to a device context
(csrc/device_once.h, DeviceCounts): built with g++ and driven on the CPU."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_causal_blockwise_gb300", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_counts_are_keyed_by_device_and_context(tmp_path):
    exe = tmp_path / "device_counts_check"
    src = os.path.join(ROOT, "tests", "host", "device_counts_check.cc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + CSRC, src, "-o", str(exe), "-lpthread"],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


def test_no_launcher_keeps_a_process_wide_answer():
    """The occupancy calculator is asked in one place, which keeps its answers by device context."""
    for name in os.listdir(CSRC):
        text = open(os.path.join(CSRC, name)).read()
        assert not re.search(r"static\s+std::atomic", text), name
        if "cudaOccupancy" in text:
            assert name == "api.cu", f"{name} asks the occupancy calculator itself"
