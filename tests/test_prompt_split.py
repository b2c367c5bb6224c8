"""The prompt attention's work split, replayed on the CPU (no device)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_every_block_goes_to_one_cta(tmp_path):
    exe = tmp_path / "prompt_split_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "transformer_layer_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "prompt_split_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_every_block_goes_to_one_cta_in_lanes(tmp_path):
    exe = tmp_path / "prompt_lanes_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "transformer_layer_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "prompt_lanes_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout
