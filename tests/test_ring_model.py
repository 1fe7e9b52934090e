"""The ring of shared-memory stages after a wait that gave up, followed on the host:
a kernel may not end while one of its copies is in flight, so its drain has to wait
for the last copy of each stage and for nothing else."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "top_routing_expert_moe_gb300", "csrc")


def test_a_drain_waits_for_the_copies_in_flight(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "ring_model")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "ring_model.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
