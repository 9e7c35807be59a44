"""The host side of the gated recurrence and the block norm (csrc/block_plan.cpp) built with the address
and undefined-behaviour sanitizers and driven through sizes at and past every limit and random argument
structures (tests/sanitize/block_driver.cpp). Plain C++: no GPU, no HIP."""
import os
import shutil

import pytest

from test_host_sanitize import ROOT, _build, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_block_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    exe = _build(tmp_path, [os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp"),
                            os.path.join(ROOT, "bidirectional_selective_scan_amd", "csrc", "block_plan.cpp")],
                 "block_driver")
    r = _run(exe)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "block driver ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
