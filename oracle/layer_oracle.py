"""CPU oracle of the feed-forward layers and their 8-bit checkpoints (NumPy,
float64); test infrastructure only.

Holds the definitions that include/sm.h states for sm_act8_pack /
sm_act8_unpack, sm_linear, sm_gated and their backward passes.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf, erfc, expit

BLOCK = 32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def round_bf16(x):
    """float64 -> the nearest bf16 value (ties to even), for values that float32 holds exactly
    or that are far from a tie; as float64."""
    u = np.asarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


# ---------------------------------------------------------------- 8-bit checkpoints

def code_values():
    """The value of each of the 256 e4m3 codes (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(s == 1, -v, v)


def act8_pack(x):
    """(codes, scales) as uint8: [T, d] and [T, ceil(d / 32)] of float64 x [T, d]."""
    T, d = x.shape
    nb = -(-d // BLOCK)
    codes = np.zeros((T, d), np.uint8)
    scales = np.zeros((T, nb), np.uint8)
    grid = code_values()[:0x7F]   # the magnitudes, ascending
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        fin = np.isfinite(v)
        mag = np.where(fin, np.abs(v), 0.0)
        e = np.full(T, -117)
        for t in range(T):
            top = mag[t].max() if mag.shape[1] else 0.0
            while top > 448.0 * 2.0 ** e[t]:
                e[t] += 1
        scales[:, b] = e + 127
        q = mag / 2.0 ** e[:, None]
        hi = np.clip(np.searchsorted(grid, q), 0, len(grid) - 1)
        lo = np.maximum(hi - 1, 0)
        up, down = grid[hi] - q, q - grid[lo]
        c = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
        c = np.where(grid[hi] == q, hi, c)
        c = np.where(e[:, None] == 120, np.minimum(c, 0x77), c)   # 256 * 2^120 is infinite
        c = np.where(np.signbit(v), c | 0x80, c)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(fin, c, 0x7F)
    return codes, scales


def act8_unpack(codes, scales):
    d = codes.shape[1]
    s = 2.0 ** (scales.astype(np.float64) - 127)
    return code_values()[codes] * np.repeat(s, BLOCK, 1)[:, :d]


# ---------------------------------------------------------------- activations

def act(name, z):
    if name == "relu":
        return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0))
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return z * 0.5 * erfc(-z / np.sqrt(2.0))
    if name == "gelu_tanh":   # (1 + tanh(u)) / 2, without its cancellation at negative u
        return z * expit(2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
    return z


def slope(name, z):
    if name == "relu":
        return np.where(np.isnan(z), z, (z > 0).astype(np.float64))
    if name == "silu":
        return expit(z) * (1 + z * expit(-z))
    if name == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2.0))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        c = 2 * np.sqrt(2 / np.pi)
        u = c * (z + 0.044715 * z ** 3)
        return expit(u) * (1 + z * expit(-u) * c * (1 + 3 * 0.044715 * z * z))
    return np.ones_like(z)


# ---------------------------------------------------------------- layers

def linear(x, w, bias=None, name="none", residual=None):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(name, z)
    return y if residual is None else y + residual


def linear_grad(dy, x, w, bias=None, name="none", rnd=lambda v: v):
    """(dx, dw, db); rnd: the rounding of dz to the layer's type."""
    dz = dy
    if name != "none":
        z = x @ w.T
        dz = rnd(dy * slope(name, z if bias is None else z + bias))
    return dz @ w, dz.T @ x, dz.sum(0)


def gated(x, wg, wu, name="silu"):
    return act(name, x @ wg.T) * (x @ wu.T)


def gated_grad(dy, x, wg, wu, name="silu", rnd=lambda v: v):
    """(dx, dwg, dwu)."""
    a, b = x @ wg.T, x @ wu.T
    da, db = rnd(dy * b * slope(name, a)), rnd(dy * act(name, a))
    return da @ wg + db @ wu, da.T @ x, db.T @ x
