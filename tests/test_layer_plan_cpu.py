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
                   '  out[0] = p.mi; out[1] = p.splits; out[2] = p.cut;\n}\n'
                   'extern "C" int few(int kind, int b, int T, int n, int d, int w, int x) {\n'
                   f'  return sm::takes_few(kind, b, T, n, d, w, x, {CUS});\n}}\n')
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


# Where one kernel takes at least a ninth longer than the other, as measured (us by the kernel for
# few tokens, by tiles).
FASTER = [("bf16", LINEAR, 1, 4096, 11008, 20.5, 30.7), ("bf16", LINEAR, 17, 11008, 4096, 28.5, 34.1),
          ("bf16", LINEAR, 32, 4096, 11008, 34.8, 29.4), ("bf16", GATED, 1, 4096, 11008, 34.1, 41.1),
          ("bf16", GATED, 24, 4096, 11008, 45.9, 40.3), ("bf16", GATED, 32, 4096, 11008, 49.2, 41.1),
          ("bf16", GATED, 24, 11008, 4096, 44.9, 50.3), ("bf16", LINEAR, 32, 1280, 5120, 9.7, 13.2),
          ("bf16", LINEAR, 16, 11008, 512, 21.7, 19.2), ("bf16", LINEAR, 32, 11008, 512, 30.8, 19.3),
          ("bf16", GATED, 1, 11008, 512, 25.0, 20.6), ("bf16", GATED, 32, 11008, 512, 40.8, 21.2),
          ("bf16", GATED, 24, 4096, 64, 15.5, 12.2), ("bf16", GATED, 32, 768, 2304, 5.4, 9.5),
          ("bf16", GATED, 24, 3416, 1280, 13.6, 16.9), ("bf16", LINEAR, 8, 11008, 64, 17.7, 14.8),
          ("f32", LINEAR, 32, 4096, 11008, 67.2, 112.0), ("f32", GATED, 32, 4096, 11008, 104.5, 163.4),
          ("f32", GATED, 24, 11008, 512, 89.2, 58.9),
          ("f32", LINEAR, 1, 11008, 512, 31.1, 56.7)]


@pytest.mark.parametrize("dt,kind,T,d,n,few,tiles", FASTER)
def test_few_tokens_take_the_faster_kernel(rules, dt, kind, T, d, n, few, tiles):
    bf16 = dt == "bf16"
    assert max(few, tiles) >= min(few, tiles) * 10 / 9
    assert bool(rules.few(kind, bf16, T, n, d, 1, 1)) == (few < tiles)
    # weights that would have to be laid out for the tiles, tokens past the kernel's, other products
    assert rules.few(kind, bf16, T, n, d, 0, 1) and not rules.few(kind, bf16, 33, n, d, 0, 0)
    assert not rules.few(SLOPE, bf16, T, n, d, 1, 1) and not rules.few(GATED_SLOPE, bf16, T, n, d, 0, 0)
