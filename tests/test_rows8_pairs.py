"""Which kernel and how many parts a product in 8 bits takes, over a grid of sizes: every
pair is among the cases that are compared on the GPU."""
import os
import subprocess

import _rows8_cases
import _rows8_pairs
from test_rows8_plan import ROOT, pytestmark  # noqa: F401


def labels(exe, sizes):
    text = "\n".join(f"{E} {R} {N} {K} {int(whole)}" for E, R, N, K, whole in sizes)
    for line in subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.splitlines():
        kind, splits, parts, chunks, pack = line.split()
        yield f"{kind} {splits}" + (f" {parts} {chunks}" if kind == "few" else "") + (" packed" if pack == "1" else "")


def steps(lo, hi, factor):
    v = float(lo)
    while v <= hi:
        yield int(v)
        v *= factor


def test_every_pair_has_a_case(tmp_path):
    exe, csrc, san = str(tmp_path / "i8_plan"), os.path.join(ROOT, "bit_moe_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-o", exe,
                    *(os.path.join(csrc, f) for f in ("experts_i8_plan.cpp", "experts_plan.cpp", "plan.cpp")),
                    os.path.join(san, "hip_standin.cpp"), os.path.join(san, "i8_plan_main.cpp")], check=True)
    cases = _rows8_cases.I8 + _rows8_pairs.I8
    sizes = [(len(n), sum(n), N, K, place % 16 == 0 and K % 16 == 0) for _, n, N, K, place in cases]
    assert list(labels(exe, sizes)) == [c[0] for c in cases]
    grid = [(E, R, N, k, whole) for E in (1, 3, 8, 64, 256) for R in steps(1, 200000, 1.37) for N in steps(1, 20000, 1.41)
            for K in steps(16, 131071, 1.33) for whole, k in ((True, K // 16 * 16), (False, K | 1), (False, K // 16 * 16))]
    assert set(labels(exe, grid)) <= {c[0] for c in cases}
