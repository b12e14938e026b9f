"""How the feed-forward layers' products are launched, from the library's own
rules (csrc/layer_plan.hpp, compiled by itself): the GPU tests' shapes reach
every way, and the rules give plans that the kernels can run."""
import ctypes
import os
import subprocess

import pytest

from matrix_aware_optimizer_momentum_amd import build_lib

CUS = 256   # of an MI355X
LINEAR, SLOPE, GATED, GATED_SLOPE, DX, DW = range(6)


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plan")
    src = folder / "plan.cpp"
    src.write_text('#include "layer_plan.hpp"\n'
                   'extern "C" void plan(int kind, int b, int M, int N, int K, int parts, int cus, '
                   'int* out) {\n'
                   '  const sm::Plan p = sm::plan_product(kind, b, M, N, K, parts, cus);\n'
                   '  out[0] = p.mi; out[1] = p.splits; out[2] = p.cut;\n}\n')
    lib = folder / "plan.so"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC",
                    f"-I{build_lib.CSRC}", str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def plan(rules, kind, bf16, M, N, K, parts=1):
    out = (ctypes.c_int * 3)()
    rules.plan(kind, int(bf16), M, N, K, parts, CUS, out)
    return tuple(out)


def way(rules, kind, bf16, M, N, K, parts=1):
    mi, splits, cut = plan(rules, kind, bf16, M, N, K, parts)
    return (64 * mi, "shares" if splits > 1 else "cut" if cut < N else "whole")


WAYS = {(64, "whole"), (128, "whole"), (128, "shares"), (256, "whole"), (256, "cut")}


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", [LINEAR, SLOPE, GATED, GATED_SLOPE])
def test_curved_activations_are_tested_in_every_way(rules, kind, bf16):
    from tests.test_gpu_layer_plans import SHAPES
    small = [(150, 96, 200)]   # of tests/test_gpu_layer.py
    assert {way(rules, kind, bf16, T, n, d) for T, d, n in SHAPES + small} == WAYS


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind,parts", [(DX, 1), (DX, 2), (DW, 1), (DW, 2)])
def test_plans_are_ones_that_the_kernels_run(rules, kind, parts, bf16):
    """And those of the four other kinds: shares have stages, and only tiles of 128; a cut is at a
    whole tile and leaves columns; two weight gradients at once are not cut."""
    sizes = [1, 7, 64, 65, 200, 515, 1003, 1280, 4096, 4104, 11008]
    for k, q in ((kind, parts), (LINEAR, 1), (GATED, 1)):
        for M in sizes:
            for N in sizes:
                for K in sizes + [70001]:
                    mi, splits, cut = plan(rules, k, bf16, M, N, K, q)
                    steps = -(-K // (64 if bf16 else 32)) * (q if k == DX else 1)
                    assert mi in (1, 2, 4) and 1 <= splits <= 16
                    assert splits == 1 or (mi == 2 and 2 * splits <= steps and cut == N)
                    cols = (32 if k == GATED else 64) * mi
                    assert cut == N or (mi == 4 and 0 < cut < N and cut % cols == 0
                                        and not (k == DW and q == 2))
