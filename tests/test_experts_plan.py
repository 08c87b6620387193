"""The rule that chooses a product's kernel (experts_plan.cpp), on the CPU: what
it takes against measured times, and that the cases which are compared with
float64 on the GPU reach every kernel."""
import os
import shutil
import subprocess

import pytest

import _experts_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORWARD, DX, DW = 0, 1, 2

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                                reason="g++ or the HIP runtime headers not available")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(layout, E, R, N, K, whole, low) of experts of N x K on 256 compute
    units: (kernel, parts of the contraction, few rows' parts and chunks)"""
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    csrc, san = os.path.join(ROOT, "bit_moe_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-o", exe,
                    os.path.join(csrc, "experts_plan.cpp"), os.path.join(csrc, "plan.cpp"),
                    os.path.join(san, "hip_standin.cpp"), os.path.join(san, "plan_main.cpp")], check=True)

    def ask(layout, E, R, N, K, whole=True, low=0):
        cols, contraction = (K, N) if layout == DX else (N, K)
        out = subprocess.run([exe], input=f"{layout} {E} {R} {cols} {contraction} {int(whole)} {low}\n", check=True,
                             capture_output=True, text=True).stdout.split()
        return out[0], int(out[1]), int(out[2]), int(out[3])
    return ask


# Measured, us, bfloat16, rows not on 16 bytes: the any-alignment kernel with the contraction in 1, 2, 4, 8, 16 parts,
# and the few-rows kernel with 1, 2, 4
ANY = [(FORWARD, 1, 2049, 7167, (119.4, 68.1, 40.9, 26.9, 23.0), (28.4, 28.2, 22.4)),
       (FORWARD, 4, 2049, 7167, (118.6, 68.1, 41.0, 27.6, 23.0), (32.9, 37.5, 37.1)),
       (FORWARD, 16, 2049, 7167, (119.0, 67.5, 41.4, 27.6, 23.5), (48.3, 69.7, 91.2)),
       (FORWARD, 64, 2049, 7167, (128.8, 74.5, 46.3, 31.0, 27.8), (113.8, 170.1, 262.3)),
       (FORWARD, 512, 2049, 7167, (143.1, 86.9, 63.6, 74.0, 79.4), ()),
       (FORWARD, 2048, 2049, 7167, (164.8, 181.3, 165.4, 172.7, 275.7), ()),
       (FORWARD, 8192, 2049, 7167, (453.4, 511.0, 578.1, 723.7, 1033.0), ()),
       (FORWARD, 16384, 4097, 1023, (299.7, 572.3, 871.2), ()),
       (FORWARD, 1, 16383, 4097, (71.1, 45.8, 37.3, 43.8, 56.3), (57.1, 61.2, 65.9)),
       (FORWARD, 4, 16383, 4097, (70.5, 44.9, 35.9, 42.7, 56.5), (67.6, 81.0, 109.1)),
       (FORWARD, 1, 513, 7167, (114.1, 64.3, 37.7, 24.6, 18.9), (27.9, 16.9, 12.1)),
       (FORWARD, 12, 513, 7167, (114.4, 64.7, 38.0, 25.3, 20.0), (42.6, 33.2, 28.2)),
       (FORWARD, 24, 513, 1001, (21.8, 17.4, 14.0), (11.7, 11.2, 11.5)),
       (DX, 16, 2049, 7167, (136.4, 78.1, 49.7, 35.2), ()),
       (DX, 512, 2049, 7167, (149.5, 101.4, 87.1, 97.5), ()),
       (DX, 8192, 2049, 7167, (473.9, 719.0, 913.0, 1321.4), ()),
       (DX, 1, 513, 7167, (32.1, 24.5), ()),
       (DX, 200, 8191, 8191, (542.2, 288.0, 171.1, 131.9, 136.2), ()),
       (DW, 512, 2049, 7167, (84.0, 106.1), ()),
       (DW, 2048, 2049, 7167, (327.3, 298.8, 294.9, 408.3), ()),
       (DW, 8192, 2049, 7167, (1314.4, 1103.5, 989.7, 1019.9, 1193.3), ()),
       (DW, 8192, 257, 263, (718.3, 364.8, 193.1, 100.0, 59.0), ()),
       (DW, 16384, 4097, 1023, (2020.5, 1234.7, 800.2, 643.7, 651.1), ())]


@pytest.mark.parametrize("layout,R,N,K,parts,few", ANY)
def test_rows_of_any_alignment(plan, layout, R, N, K, parts, few):
    """A cost in three constants meets the best of these within 40%."""
    kind, splits, p, _ = plan(layout, 1, R, N, K, whole=False)
    assert kind in ("any", "few")
    at = [1, 2, 4, 8, 16]
    took = few[at.index(p)] if kind == "few" else parts[at.index(splits)]
    assert took <= 1.4 * min(parts + few), (kind, splits, p, took)


def whole(N, K, place, layout):
    """Every row of the operands on 16 bytes (dense ones, from `place` on)."""
    return place % 8 == 0 and K % 8 == 0 and (N % 8 == 0 or layout == FORWARD)


def name(took):
    kind, splits, parts, chunks = took
    return f"{kind} {splits}" + (f" {parts} {chunks}" if kind == "few" else "")


@pytest.mark.parametrize("layout,list_of", [(FORWARD, "FORWARD"), (DX, "DX"), (DW, "DW")])
def test_cases_reach_every_kernel(plan, layout, list_of):
    """The sizes that are compared with float64 take the kernels that they are
    listed for, and no kernel that can be launched is missing."""
    listed = getattr(cases, list_of)
    for label, counts, N, K, place in listed:
        took = plan(layout, len(counts), sum(counts), N, K, whole(N, K, place, layout))
        assert name(took) == label, (counts, N, K, place, name(took))
    kinds = {"256x256", "128x128", "any"} | ({"128x256", "64x128"} if layout != DW else set())
    few = {f"few 1 {p} {c}" for p in (1, 2, 4) for c in (1, 4)} if layout == FORWARD else set()
    labels = {c[0] for c in listed}
    assert {c.split()[0] for c in labels} == kinds | ({"few"} if few else set())
    assert few <= labels
    assert {int(c.split()[1]) for c in labels} == {1, 2, 4, 8, 16}         # of each join, too
    # groups of several experts, an empty one among them, in every kind
    assert {c[0].split()[0] for c in listed if len(c[1]) > 1 and 0 in c[1]} >= kinds


def test_backward_cases_reach_every_kernel(plan):
    for dx, dw, T, N, K, pad, place in cases.BACKWARD:
        on16 = lambda layout: whole(N, K, place, layout) and pad % 8 == 0  # noqa: E731
        for layout, label in ((DX, dx), (DW, dw)):
            took = plan(layout, 1, T, N, K, on16(layout), low=8)
            assert name(took) == label, (layout, T, N, K, name(took))
    assert {c[0].split()[0] for c in cases.BACKWARD} == {"256x256", "128x256", "128x128", "64x128", "any"}
    assert {c[1].split()[0] for c in cases.BACKWARD} == {"256x256", "128x128", "any"}
    for i in (0, 1):
        assert {int(c[i].split()[1]) for c in cases.BACKWARD} == {1, 2, 4, 8, 16}
