"""The rule that chooses the kernel of a product in 8 bits (experts_i8_plan.cpp),
on the CPU: what it takes against measured times, and that the cases which are
compared on the GPU reach every kernel."""
import os
import shutil
import subprocess

import pytest

import _rows8_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                                reason="g++ or the HIP runtime headers not available")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "i8_plan")
    csrc, san = os.path.join(ROOT, "bit_moe_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-o", exe,
                    *(os.path.join(csrc, f) for f in ("experts_i8_plan.cpp", "experts_plan.cpp", "plan.cpp")),
                    os.path.join(san, "hip_standin.cpp"), os.path.join(san, "i8_plan_main.cpp")], check=True)

    def ask(E, R, N, K, whole=True):
        out = subprocess.run([exe], input=f"{E} {R} {N} {K} {int(whole)}\n", check=True, capture_output=True, text=True).stdout
        kind, splits, parts, chunks, pack = out.split()
        return f"{kind} {splits}" + (f" {parts} {chunks}" if kind == "few" else "") + (" packed" if pack == "1" else "")
    return ask


# Measured, us, bfloat16 outputs, several calls in a row; "" in a key: any number of parts
MEASURED = [(1, 8192, 4096, 7168, {"256x256 1": 188.6, "128x256 1": 201.7, "128x128 1": 210.2, "64x128 1": 280.5}),
            (1, 8192, 8192, 8192, {"256x256 1": 390.7, "128x256 1": 462.9, "128x128 1": 530.3, "64x128 1": 688.1}),
            (32, 32768, 7168, 2048, {"256x256 1": 469.0, "128x256 1": 591.8, "128x128 1": 609.4, "64x128 1": 783.7}),
            (256, 16384, 2048, 7168, {"256x256 1": 826.9, "128x256 1": 682.2, "128x128 1": 709.7, "64x128 1": 839.6}),
            (256, 2048, 4096, 7168, {"128x256 1": 1229.1, "128x128 1": 1253.6, "64x128 1": 1226.8, "few 1 1 1": 1729.3}),
            (256, 8, 4096, 7168, {"few 1 1 1": 51.9, "few 1 2 1": 57.7, "few 1 4 1": 75.9, "64x128 1": 44.7, "64x128 2": 50.9,
                                  "128x128 2": 51.5}),
            (256, 16, 2048, 2048, {"few 1 1 1": 15.1, "few 1 2 1": 21.2, "64x128 1": 14.3, "64x128 2": 18.3}),
            (1, 512, 2048, 7168, {"256x256 4": 40.6, "128x128 1": 29.8, "128x128 2": 28.7, "64x128 1": 23.7, "64x128 2": 25.3,
                                  "128x256 4": 31.5}),
            (1, 1024, 2048, 7168, {"256x256 4": 46.0, "128x128 1": 30.7, "64x128 1": 24.7, "64x128 2": 36.2, "128x256 4": 37.4}),
            (1, 2048, 2048, 7168, {"256x256 4": 61.0, "128x128 1": 34.3, "64x128 1": 38.5, "128x256 1": 42.2}),
            (1, 8192, 2048, 7168, {"256x256 1": 91.9, "128x256 1": 109.3, "128x128 1": 117.6, "64x128 1": 158.3}),
            (1, 64, 2048, 7168, {"64x128 8": 16.3, "64x128 4": 16.4, "128x128 8": 17.7, "few 1 1 1": 17.3, "few 1 2 1": 31.7}),
            (1, 1, 16384, 4096, {"few 1 1 1": 17.7, "few 1 2 1": 19.7, "few 1 4 1": 25.3, "64x128 1": 21.6, "64x128 2": 21.3}),
            (8, 666, 1001, 2047, {"any 1": 38.2, "any 2": 35.7, "any 4": 33.7, "any 8": 41.4, "64x128 1 packed": 24.3}),
            (1, 8192, 2049, 7167, {"any 1": 270.1, "any 2": 373.9, "128x128 1 packed": 161.0}),
            (1, 16, 2049, 7167, {"any 8": 26.4, "any 16": 26.1, "few 1 1 1": 31.4, "few 1 2 4": 44.5, "64x128 8 packed": 26.4}),
            (63, 42, 7632, 1805, {"any 1": 94.3, "any 2": 103.8, "few 1 1 1": 152.0})]


@pytest.mark.parametrize("E,R,N,K,took", MEASURED, ids=str)
def test_the_rule_meets_the_measured(plan, E, R, N, K, took):
    """What the rule takes is within 15% of the best that was measured."""
    label = plan(E, R, N, K, K % 16 == 0)
    assert label in took and took[label] <= 1.15 * min(took.values()), (label, took)


def test_cases_reach_every_kernel(plan):
    """The sizes that are compared on the GPU take the kernels that they are listed
    for, and no kernel that can be launched is missing."""
    for label, counts, N, K, place in cases.I8:
        assert plan(len(counts), sum(counts), N, K, place % 16 == 0 and K % 16 == 0) == label, (counts, N, K, place)
    labels = {c[0] for c in cases.I8}
    assert {c.split()[0] for c in labels} == {"256x256", "128x256", "128x128", "64x128", "any", "few"}
    assert {f"few 1 {p} {c}" for p in (1, 2, 4) for c in (1, 4)} <= labels
    assert {int(c.split()[1]) for c in labels} == {1, 2, 4, 8, 16}
    assert {c.split()[0] for c in labels if "packed" in c} == {"256x256", "128x128", "64x128"}
    # groups of several experts, an empty one among them, in every kind, packed too
    for kind in {c.split()[0] + (" packed" if "packed" in c else "") for c in labels}:
        assert any(0 in c[1] for c in cases.I8 if c[0].split()[0] + (" packed" if "packed" in c[0] else "") == kind), kind


def test_nothing_is_laid_out_past_4_gibibytes(plan):
    assert plan(256, 64, 4096, 7167, False).split()[0] in ("any", "few")
    assert "packed" in plan(64, 65536, 2048, 7167, False) and "packed" not in plan(256, 65536, 4096, 7167, False)
    assert "packed" not in plan(64, 65536, 2048, 7168, False)            # whole rows, whose addresses are odd
