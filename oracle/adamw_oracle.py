"""CPU oracle of the AdamW operators (NumPy, float64); test infrastructure only.

Holds the definitions that include/sm.h states for sm_adamw, sm_grad_norm and
sm_state8_pack / sm_state8_unpack: moments and weights in float64 from the
stored inputs, the random bits and the 8-bit grids.  Rounded results come
with the interval that a float32 evaluation may round from.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256
M32 = 0xFFFFFFFF


def f32(v) -> float:
    return float(np.float32(v))


# ---------------------------------------------------------------- random bits

def mix(x):
    """The 32-bit mixing, on uint64 arrays or ints holding 32-bit values."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & M32
    x = x ^ (x >> 15)
    x = (x * 0x85A308D3) & M32
    return x ^ (x >> 16)


def _word(key: int, word: int) -> int:
    return mix(((key ^ word) + 0x9E3779B9) & M32)


def random_bits(seed: int, t: int, index: int, entries: np.ndarray):
    """(r, r_w): 32 random bits per entry for the states, 16 for the weights."""
    key = 0
    for word in (seed & M32, seed >> 32, t & M32, t >> 32, index):
        key = _word(key, word)
    r = np.empty(len(entries), np.uint64)
    for hi in np.unique(entries >> 32):
        sel = (entries >> 32) == hi
        k = _word(key, int(hi))
        r[sel] = mix((entries[sel].astype(np.uint64) & np.uint64(M32)) ^ np.uint64(k))
    return r, mix(r ^ np.uint64(0x9E3779B1)) & np.uint64(0xFFFF)


# ---------------------------------------------------------------- 8-bit grids

KINDS = {"m": (3, -6, 8, 448.0), "v": (2, -14, 15, 57344.0)}   # mantissa, lowest, top, largest


def scale_of(amax: float, kind: str) -> float:
    """The smallest power of two (at least 2^-126) with amax <= largest * scale."""
    _, _, _, largest = KINDS[kind]
    e = -126
    if amax > 0:
        e = max(-126, int(np.floor(np.log2(amax))) - 17)
        while largest * 2.0 ** e < amax:
            e += 1
    return 2.0 ** e


def scales(x: np.ndarray, kind: str) -> np.ndarray:
    """Scale of every block of x (flat), over its finite entries."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    return np.array([scale_of(a[i:i + BLOCK].max(), kind) for i in range(0, len(a), BLOCK)])


def per_entry(s: np.ndarray, n: int) -> np.ndarray:
    return np.repeat(s, BLOCK)[:n]


def step_of(x: np.ndarray, kind: str) -> np.ndarray:
    """Distance between neighbouring codes at magnitude x (in scaled units)."""
    keep, lowest, _, _ = KINDS[kind]
    e = np.frexp(x)[1] - 1
    return np.ldexp(1.0, np.maximum(np.where(x > 0, e, lowest), lowest) - keep)


def to_grid(x: np.ndarray, kind: str, u=None) -> np.ndarray:
    """Scaled magnitudes on the codes' grid: floor(x / step + u) steps, or to
    nearest even without u."""
    q = step_of(x, kind)
    return (np.rint(x / q) if u is None else np.floor(x / q + u)) * q


def pack(x: np.ndarray, kind: str):
    """(code values, scales) of finite float32 states, to nearest."""
    s = scales(x, kind)
    a = np.abs(x) / per_entry(s, len(x))
    c = to_grid(a, kind)
    if kind == "v":
        c = np.where(x > 0, np.maximum(c, 2.0 ** -16), 0.0)
    return np.copysign(c, x) if kind == "m" else c, s


# ---------------------------------------------------------------- the step

def moments(grads, m, v, c1: dict, gscale=1.0):
    """(g, m, v) of a step in float64; grads: [M, n] of stored values."""
    b1, b2 = f32(c1["beta1"]), f32(c1["beta2"])
    with np.errstate(all="ignore"):
        g = np.asarray(grads, np.float64).sum(0) * (f32(gscale) / len(grads))
        return g, b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g


def weights(w, m, v, t: int, c1: dict, wd=0.0, lr_mult=1.0, lr_scale=1.0):
    """(new weights, size of the step's change) in float64."""
    b1, b2 = f32(c1["beta1"]), f32(c1["beta2"])
    lr = f32(c1["lr"]) * f32(lr_mult) * f32(lr_scale)
    with np.errstate(all="ignore"):
        den = np.sqrt(v / (1 - b2 ** t)) + f32(c1["eps"])
        d = lr * (m / (1 - b1 ** t)) / den
        return w * (1 - lr * f32(wd)) - d, np.abs(d)


def grad_norm(sets, scale: float, max_norm: float):
    """sets: [(M, [grads [M, n] ...]) ...] -> (norm, factor)."""
    s = 0.0
    with np.errstate(all="ignore"):
        for M, grads in sets:
            for g in grads:
                mean = np.asarray(g, np.float64).sum(0) / M
                s += float(np.sum(mean * mean))
        norm = abs(scale) * np.sqrt(s)
    if not np.isfinite(norm):
        return norm, float("nan")
    return norm, scale * min(1.0, max_norm / (norm + 1e-6))
