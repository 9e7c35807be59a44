"""The windows of the decays' gradient, host side, under the address and undefined-behaviour sanitizers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_windows_under_sanitizers(tmp_path):
    exe = tmp_path / "driver"
    src = [os.path.join(ROOT, "tests", "sanitize", "linattn_windows_driver.cpp"),
           os.path.join(ROOT, "bidirectional_selective_scan_amd", "csrc", "linattn_plan.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
                    "-I", os.path.join(ROOT, "include"), "-o", str(exe)] + src, check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
