"""Refusals of the feed-forward layers' calls that their queries cannot make: of
the workspace, and of buffers between a matrix's rows (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from matrix_aware_optimizer_momentum_amd import _binding as B
from oracle import layer_oracle as L
from tests.test_layer_cpu import ARG, CALLS, OK, WORKSPACE, _layer, _refusal

# every operand is laid out, every product has scratch of its own
SIZES = dict(T=50, d=17, n=33, ldx=17, ldw=17, ldw2=17, ldr=33, ldy=33, lddy=33, lddx=17, lddw=17,
             lddw2=17)
BUFFERS = {"linear": ("x", "w", "bias", "residual", "y"), "gated": ("x", "w", "w2", "y"),
           "linear_grad": ("x", "w", "bias", "dy", "dx", "dw", "dbias"),
           "gated_grad": ("x", "w", "w2", "dy", "dx", "dw", "dw2")}


@pytest.mark.parametrize("call,name", [(c, b) for c in CALLS for b in BUFFERS[c]])
def test_a_workspace_over_a_buffer_is_refused(call, name):
    lib = B.lib()
    l, need = _layer(**SIZES), ctypes.c_size_t(0)
    assert getattr(lib, f"sm_{call}_ws")(ctypes.byref(l), ctypes.byref(need)) == OK
    assert need.value > 0
    at = getattr(l, name)
    last = at + 4 * (33 if "bias" in name else 17 * 33) - 4   # of a part of the buffer
    for ws in (at, last // 256 * 256, at - (need.value - 1) // 256 * 256):
        assert getattr(lib, f"sm_{call}")(ctypes.byref(l), ws, need.value, None) == ARG, hex(ws)
        assert getattr(lib, f"sm_{call}")(ctypes.byref(l), ws, need.value - 1, None) == WORKSPACE
    assert lib.sm_last_hip_error() == 0


def test_a_workspace_over_a_checkpoint_is_refused():
    lib = B.lib()
    for at in (0xF00000, 0xF80000):
        l, need = _layer(x=None, x8=0xF00000, x8_scale=0xF80000, **SIZES), ctypes.c_size_t(0)
        assert lib.sm_gated_grad_ws(ctypes.byref(l), ctypes.byref(need)) == OK
        assert lib.sm_gated_grad(ctypes.byref(l), at, need.value, None) == ARG
    assert lib.sm_last_hip_error() == 0


@pytest.mark.parametrize("call,kw,want", [
    # 24 entries between rows of 16 that are 64 apart, and one entry into a row
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * 16), OK),
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * 40), OK),
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * 41), ARG),
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * 15), ARG),
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * (64 * 23 + 15)), ARG),
    ("linear_grad", dict(lddw=64, dbias=0x900000 + 4 * (64 * 23 + 16)), OK),
])
def test_vectors_between_rows(call, kw, want):
    assert _refusal(call, **kw) == want


def test_the_vectorised_reference_of_checkpoints_is_the_oracle():
    from tests.test_gpu_act8 import pack_reference, values_of
    rng = np.random.default_rng(0)
    v = rng.standard_normal((60, 100)) * np.exp(4 * rng.standard_normal((60, 1)))
    for value in (np.inf, -np.inf, np.nan, 3.3e38, -3.4e38, 1e-38, 448.0, 0.0):
        v[rng.random(v.shape) < 0.05] = value
    v[7], v[8], v[9] = 3.4e38, 0.0, np.nan
    x = torch.from_numpy(v).float()
    codes, scales = pack_reference(x)
    want = L.act8_pack(x.double().numpy())
    np.testing.assert_array_equal(codes.numpy(), want[0])
    np.testing.assert_array_equal(scales.numpy(), want[1])
    np.testing.assert_array_equal(values_of(codes, scales, "cpu").numpy(), L.act8_unpack(*want))
