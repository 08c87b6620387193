"""The host code of the operators in 8 bits and of the block norms (validation, the
rule that chooses kernels and workspaces) under AddressSanitizer and
UndefinedBehaviorSanitizer, over sizes up to the largest a call accepts (CPU
only)."""
import os
import shutil

import pytest

from test_sanitizers import ENV, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP runtime headers not available")
def test_rows8_host_code_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "rows8_san")
    csrc = os.path.join(ROOT, "bit_moe_amd", "csrc")
    san = os.path.join(ROOT, "tests", "sanitize")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-o", exe,
                    *(os.path.join(csrc, f) for f in ("rows8.cpp", "norm.cpp", "experts_i8_plan.cpp", "experts_plan.cpp", "plan.cpp")),
                    os.path.join(san, "hip_standin.cpp"), os.path.join(san, "rows8_main.cpp")])
    assert rc == 0, out
    rc, out = _run([exe], ENV)
    assert rc == 0 and "rows8 sanitizer driver: ok" in out, out
    assert "runtime error" not in out and "ERROR: AddressSanitizer" not in out, out
