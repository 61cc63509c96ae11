"""CPU check of the rule that says which kernel a call of moe_grouped_gemm_mxfp4 takes (the launch's own
host code, built with g++): the problems of the GPU tests reach every kernel that is compiled."""

import os
import re
import shutil
import subprocess

import pytest

from routed_moe_layer_amd import build as b
from tests.mxfp4_kernels import CUS, PROBLEMS, WIDE_WEIGHTS, sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """kernels of [(R, E, Nw, KB, x_rows, gathered)]: (rows, waves, workgroups a CU, wide, direct)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("rule") / "rule"
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror", f"-I{b.CSRC}",
                    os.path.join(ROOT, "tests", "c", "mxfp4_rule.cpp"), "-o", str(exe)], check=True)

    def ask(problems):
        lines = "".join(" ".join(str(int(v)) for v in (*p, CUS)) + "\n" for p in problems)
        out = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return ask


def test_the_problems_reach_the_kernels_that_they_are_named_for(rule):
    for situ in (False, True):
        asked = []
        for kernel in PROBLEMS:
            R, E, N, K, x_rows = sizes(kernel, situ)
            asked.append((R, E, 2 * N if situ else N, K // 2, x_rows, kernel[4] != "plain"))
        for kernel, got in zip(PROBLEMS, rule(asked)):
            assert got == (*kernel[:3], kernel[3], kernel[4] == "direct"), (kernel, situ)
    asked = [(R, E, 2 * N, K // 2, R, False) for R, E, N, K in WIDE_WEIGHTS.values()]
    for kernel, got in zip(WIDE_WEIGHTS, rule(asked)):
        assert got == (*kernel[:4], False), kernel


def test_they_reach_every_kernel(rule):
    with open(os.path.join(b.CSRC, "grouped_mxfp4.hip")) as fh:
        launches = re.findall(r"launch_mx_mid<SITU, (\w+), (\d+), (\d+), (\d+)>\(a, s", fh.read())
    tiles = {(int(r), int(w), int(n), wide == "true") for wide, r, w, n in launches}
    assert len(tiles) == len(launches) == 7
    want = {(*t, how) for t in tiles for how in ("plain", "list", "direct")}
    want |= {(256, 4, 1, False, how) for how in ("plain", "gathered")}
    assert set(PROBLEMS) | set(WIDE_WEIGHTS) == want


def test_a_list_that_does_not_fit_is_not_made(rule):
    """Behind 128-row tiles and 50 experts' prefix sums 1700 entries fit and 1710 do not."""
    assert rule([(1700, 50, 1024, 144, 600, True), (1710, 50, 1024, 144, 600, True)]) == [
        (128, 8, 1, 0, 0), (128, 8, 1, 0, 1)]
