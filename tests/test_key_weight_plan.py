"""How mla_key_weight cuts its work, on the CPU: shares neither overlap nor leave gaps, and are even."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
@pytest.mark.parametrize("args", [[], ["chunks"]])
def test_shares(tmp_path, args):
    exe = tmp_path / "check"
    csrc = os.path.join(os.path.dirname(HERE), "attention_prologue_kv_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-x", "c++", "-I", csrc, os.path.join(HERE, "key_weight_plan_check.cpp"), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)] + args, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout
