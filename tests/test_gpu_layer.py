"""The feed-forward layers and their 8-bit checkpoints on the GPU, against the
float64 oracle.

Whole numbers.  With small whole numbers as inputs, and act none or relu,
every product and every float32 sum is exact (all partial sums stay below
2^24) and what is rounded to bf16 is rounded from the exact value: results
have to equal the oracle's bit for bit, whatever the order of the sums.

Other numbers.  A float32 sum of K products is off by at most K * 2^-23 of the
sum of the products' magnitudes (2^-24 for an addition to nearest, twice that
where the matrix cores cut bits off).  An activation moves by at most 1.13
times that (the largest slope of all of them), plus its own evaluation's
error: 2^-20 of |z| + |value| covers its exp, division and erfc (each a few
2^-24 of their value, |z| 2^-24 for exp's argument).  A result is rounded by
half a step: 2^-8 of the value (bf16) or 2^-24 (float32); dz, rounded too, by
as much ahead of the sums that it enters.
"""
import gc

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm
from oracle import layer_oracle as L

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
ACT = {"none": sm.ACT_NONE, "relu": sm.ACT_RELU, "silu": sm.ACT_SILU, "gelu": sm.ACT_GELU,
       "gelu_tanh": sm.ACT_GELU_TANH}


def np64(t):
    return t.detach().double().cpu().numpy()


def rnd(dt):
    return L.round_bf16 if dt == "bf16" else lambda v: np.asarray(v, np.float32).astype(np.float64)


class Guarded:
    """A [rows, cols] tensor inside a larger buffer: `shift` entries off a 256-byte boundary, rows
    `cols + gap` apart, sentinels (NaN) everywhere else."""

    MARK = 0xFF   # NaN in both types

    def __init__(self, value, dt, shift=0, gap=0):
        rows, cols = value.shape
        ld = cols + gap
        dtype = DT[dt]
        size = torch.empty(0, dtype=dtype).element_size()
        n = 256 + shift + rows * ld + 256
        self.raw = torch.full((n * size,), self.MARK, dtype=torch.uint8, device="cuda")
        flat = self.raw.view(dtype)
        self.t = flat[256 + shift:256 + shift + rows * ld].view(rows, ld)[:, :cols]
        self.t.copy_(torch.from_numpy(np.ascontiguousarray(value)).to(dtype))
        inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        inside[256 + shift:256 + shift + rows * ld].view(rows, ld)[:, :cols] = True
        self.outside = ~inside.repeat_interleave(size)

    def check(self, what):
        assert bool((self.raw[self.outside] == self.MARK).all()), f"{what}: written outside"


def whole(rng, shape, top):
    return rng.integers(-top, top + 1, shape).astype(np.float64)


# (T, d, n): one token, odd sizes, edges of tiles of 32, 64, 128 and 256 and of k steps, more rows
# than columns and the reverse
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 130, 257), (3, 8, 16), (7, 33, 31), (16, 96, 200), (17, 40, 520),
          (32, 64, 64), (33, 127, 129), (64, 256, 64), (65, 72, 136), (100, 20, 300), (129, 136, 264),
          (255, 64, 40), (256, 128, 256), (257, 264, 136), (300, 520, 72), (520, 48, 48), (31, 1000, 24)]
# buffers as they come: entries off alignment, columns between rows
LAYOUTS = [(0, 0), (1, 0), (0, 8), (3, 5)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_whole_numbers_linear(gpu_lib, dt, shape, layout):
    T, d, n = shape
    rng = np.random.default_rng(T * 7 + d * 3 + n)
    x, w, bias = whole(rng, (T, d), 3), whole(rng, (n, d), 3), whole(rng, (n,), 9)
    res, dy = whole(rng, (T, n), 20), whole(rng, (T, n), 2)
    g = lambda v: Guarded(v, dt, *layout)
    X, W, R, DY = g(x), g(w), g(res), g(dy)
    Y, DX, DW = g(np.full((T, n), np.nan)), g(np.full((T, d), np.nan)), g(np.full((n, d), np.nan))
    b = torch.from_numpy(bias).to(DT[dt]).cuda()
    for name in ("none", "relu"):
        a = ACT[name]
        sm.linear(X.t, W.t, bias=b, act=a, residual=R.t, out=Y.t)
        np.testing.assert_array_equal(np64(Y.t), rnd(dt)(L.linear(x, w, bias, name, res)))
        dx, dw, db = sm.linear_grad(DY.t, X.t, W.t, bias=b, act=a, dx=DX.t, dw=DW.t)
        want = L.linear_grad(dy, x, w, bias, name, rnd(dt))
        for got, v in zip((dx, dw, db), want):
            np.testing.assert_array_equal(np64(got), rnd(dt)(v))
    assert torch.equal(sm.linear(X.t, W.t), torch.from_numpy(rnd(dt)(x @ w.T)).to(DT[dt]).cuda())
    for q, what in ((Y, "y"), (DX, "dx"), (DW, "dw"), (X, "x"), (W, "w"), (DY, "dy")):
        q.check(what)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_whole_numbers_gated(gpu_lib, dt, shape, layout):
    T, d, n = shape
    rng = np.random.default_rng(T * 5 + d * 11 + n)
    x, wg, wu = whole(rng, (T, d), 1), whole(rng, (n, d), 2), whole(rng, (n, d), 1)
    dy = whole(rng, (T, n), 1)
    g = lambda v: Guarded(v, dt, *layout)
    X, WG, WU, DY = g(x), g(wg), g(wu), g(dy)
    Y, DX = g(np.full((T, n), np.nan)), g(np.full((T, d), np.nan))
    DG, DU = g(np.full((n, d), np.nan)), g(np.full((n, d), np.nan))
    for name in ("none", "relu"):
        a = ACT[name]
        sm.gated(X.t, WG.t, WU.t, act=a, out=Y.t)
        np.testing.assert_array_equal(np64(Y.t), rnd(dt)(L.gated(x, wg, wu, name)))
        got = sm.gated_grad(DY.t, X.t, WG.t, WU.t, act=a, dx=DX.t, dwg=DG.t, dwu=DU.t)
        want = L.gated_grad(dy, x, wg, wu, name, rnd(dt))
        for q, v in zip(got, want):
            np.testing.assert_array_equal(np64(q), rnd(dt)(v))
    for q, what in ((Y, "y"), (DX, "dx"), (DG, "dwg"), (DU, "dwu"), (X, "x"), (WG, "wg"),
                    (WU, "wu"), (DY, "dy")):
        q.check(what)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", [(2900, 2904, 2888), (2883, 2901, 2897), (4200, 72, 4104), (4200, 4104, 72),
                                   (40, 4104, 4200), (200, 4101, 1003)])
def test_whole_numbers_large(gpu_lib, dt, T, d, n):
    """Enough rows and columns for the large tiles in every product; float64 on the GPU as the
    reference (whole numbers: exact there too)."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    f = lambda top, *s: torch.randint(-top, top + 1, s, generator=gen, device="cuda").to(DT[dt])
    x, wg, wu, bias, res, dy = f(1, T, d), f(2, n, d), f(1, n, d), f(9, n), f(20, T, n), f(1, T, n)
    X, G, U, BI, R, DY = (v.double() for v in (x, wg, wu, bias, res, dy))
    a, b = X @ G.T, X @ U.T

    def same(got, want):
        assert torch.equal(got, want.to(DT[dt]))

    relu = dict(act=sm.ACT_RELU)
    same(sm.linear(x, wg, bias=bias, residual=res, **relu), (a + BI).relu() + R)
    same(sm.gated(x, wg, wu, **relu), a.relu() * b)
    dz = DY * (a + BI > 0)
    dx, dw, db = sm.linear_grad(dy, x, wg, bias=bias, **relu)
    same(dx, dz @ G)
    same(dw, dz.T @ X)
    same(db, dz.sum(0))
    da, dbb = (v.to(DT[dt]).double() for v in (DY * b * (a > 0), DY * a.relu()))
    old = f(50, 2, n, d)
    new = old.clone()
    dx, _, _ = sm.gated_grad(dy, x, wg, wu, dwg=new[0], dwu=new[1], accumulate=True, **relu)
    same(dx, da @ G + dbb @ U)
    same(new[0], old[0].double() + da.T @ X)
    same(new[1], old[1].double() + dbb.T @ X)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n", [(1, 1), (255, 129), (256, 3), (257, 130), (5000, 77), (300000, 5)])
def test_bias_gradients_of_any_length(gpu_lib, dt, T, n):
    gen = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randint(-2, 3, (T, n), generator=gen, device="cuda").to(DT[dt])
    x, w = torch.zeros(T, 1, device="cuda", dtype=DT[dt]), torch.zeros(n, 1, device="cuda", dtype=DT[dt])
    old = torch.randint(-9, 10, (n,), generator=gen, device="cuda").to(DT[dt])
    _, _, db = sm.linear_grad(dy, x, w, bias=old, need_dx=False, need_dw=False)
    assert torch.equal(db, dy.double().sum(0).to(DT[dt]))
    want = (dy.double().sum(0) + old.double()).to(DT[dt])
    sm.linear_grad(dy, x, w, db=old, need_dx=False, need_dw=False, accumulate=True)
    assert torch.equal(old, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", [(5, 40, 24), (70, 130, 90), (200, 64, 300)])
def test_accumulate_and_left_out_results(gpu_lib, dt, T, d, n):
    rng = np.random.default_rng(T)
    x, wg, wu = whole(rng, (T, d), 1), whole(rng, (n, d), 2), whole(rng, (n, d), 1)
    bias, dy = whole(rng, (n,), 2), whole(rng, (T, n), 1)
    old, old_b = whole(rng, (2, n, d), 50), whole(rng, (2, n), 50)
    t = lambda v: torch.from_numpy(v).to(DT[dt]).cuda()
    X, WG, WU, BI, DY = t(x), t(wg), t(wu), t(bias), t(dy)
    # the second worker's streams: the first one's stay
    grads, grads_b, grads_u = t(old), t(old_b), t(old)
    sm.linear_grad(DY, X, WG, bias=BI, act=sm.ACT_RELU, dw=grads[1], db=grads_b[1],
                   need_dx=False, accumulate=True)
    _, dw, db = L.linear_grad(dy, x, wg, bias, "relu", rnd(dt))
    np.testing.assert_array_equal(np64(grads), rnd(dt)(old + np.stack([0 * dw, dw])))
    np.testing.assert_array_equal(np64(grads_b), rnd(dt)(old_b + np.stack([0 * db, db])))
    grads = t(old)
    got = sm.gated_grad(DY, X, WG, WU, act=sm.ACT_RELU, dwg=grads[1], dwu=grads_u[0],
                        accumulate=True)
    dx, dwg, dwu = L.gated_grad(dy, x, wg, wu, "relu", rnd(dt))
    np.testing.assert_array_equal(np64(got[0]), rnd(dt)(dx))
    np.testing.assert_array_equal(np64(grads), rnd(dt)(old + np.stack([0 * dwg, dwg])))
    np.testing.assert_array_equal(np64(grads_u), rnd(dt)(old + np.stack([dwu, 0 * dwu])))
    # one result alone
    only = sm.gated_grad(DY, X, WG, WU, act=sm.ACT_RELU, need_dw=False)
    assert torch.equal(only[0], got[0]) and only[1] is None and only[2] is None
    only = sm.linear_grad(DY, X, WG, bias=BI, act=sm.ACT_RELU, need_dx=False, need_dw=False)
    assert only[0] is None and only[1] is None
    np.testing.assert_array_equal(np64(only[2]), rnd(dt)(db))
    # onto the residual stream, in place
    y = t(whole(rng, (T, n), 9))
    want = rnd(dt)(L.linear(x, wg, None, "none", np64(y)))
    assert sm.linear(X, WG, residual=y, out=y) is y
    np.testing.assert_array_equal(np64(y), want)


# ---------------------------------------------------------------- other numbers

def sum_error(K, mags):
    return K * 2.0 ** -23 * mags


def close(got, want, bound, what):
    err = np.abs(np64(got) - want)
    worst = float(np.max(err / bound)) if err.size else 0.0
    assert np.all(err <= bound), f"{what}: {worst:.2f} times its bound"


def act_error(z, ez, scale):
    """Of scale * act(z) or scale * act'(z), z off by ez (slopes and curvatures are below 1.13)."""
    return np.abs(scale) * (1.13 * ez + 2.0 ** -20 * (1 + np.abs(z)))


@pytest.mark.parametrize("name", L.ACTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", [(1, 200, 130), (9, 33, 50), (150, 96, 200)])
def test_activations_linear(gpu_lib, T, d, n, dt, name):
    rng = np.random.default_rng(T + d)
    t = lambda v: torch.from_numpy(v).to(DT[dt]).cuda()
    # z from -9 to 9: tails of every activation too
    X, W = t(rng.standard_normal((T, d))), t(3 * d ** -0.5 * rng.standard_normal((n, d)))
    BI, R = t(rng.standard_normal(n)), t(rng.standard_normal((T, n)))
    DY = t(rng.standard_normal((T, n)))
    x, w, bias, res, dy = (np64(v) for v in (X, W, BI, R, DY))
    z = x @ w.T + bias
    ez = sum_error(d + 1, np.abs(x) @ np.abs(w).T + np.abs(bias))
    y = L.linear(x, w, bias, name, res)
    half = HALF[dt]
    ey = act_error(z, ez, 1) + 2.0 ** -23 * (np.abs(y) + np.abs(res))
    close(sm.linear(X, W, bias=BI, act=ACT[name], residual=R), y, ey * (1 + half) + half * np.abs(y), "y")
    if name == "relu":   # its slope jumps: entries near 0 are left out of the comparison
        dy = np.where(np.abs(z) <= ez, 0.0, dy)
        DY = t(dy)
    dx, dw, db = sm.linear_grad(DY, X, W, bias=BI, act=ACT[name])
    dz = dy * L.slope(name, z)
    edz = np.zeros_like(dz)
    if name != "none":
        edz = act_error(z, ez, dy)
        edz = edz * (1 + half) + half * np.abs(dz)
    for got, want, e, mags, k in (
            (dx, dz @ w, edz @ np.abs(w), (np.abs(dz) + edz) @ np.abs(w), n),
            (dw, dz.T @ x, edz.T @ np.abs(x), (np.abs(dz) + edz).T @ np.abs(x), T),
            (db, dz.sum(0), edz.sum(0), (np.abs(dz) + edz).sum(0), T)):
        e = e + sum_error(k, mags)
        close(got, want, e * (1 + half) + half * np.abs(want), "gradient")


@pytest.mark.parametrize("name", L.ACTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", [(1, 200, 130), (9, 33, 50), (150, 96, 200)])
def test_activations_gated(gpu_lib, T, d, n, dt, name):
    rng = np.random.default_rng(T + d + 1)
    t = lambda v: torch.from_numpy(v).to(DT[dt]).cuda()
    X, G = t(rng.standard_normal((T, d))), t(3 * d ** -0.5 * rng.standard_normal((n, d)))
    U, DY = t(d ** -0.5 * rng.standard_normal((n, d))), t(rng.standard_normal((T, n)))
    x, wg, wu, dy = (np64(v) for v in (X, G, U, DY))
    a, b = x @ wg.T, x @ wu.T
    ea, eb = (sum_error(d, np.abs(x) @ np.abs(v).T) for v in (wg, wu))
    half = HALF[dt]
    h = L.act(name, a)
    fine = 2.0 ** -22   # the products of the epilogue
    ey = act_error(a, ea, np.abs(b) + eb) + np.abs(h) * eb + fine * np.abs(h * b)
    y = h * b
    close(sm.gated(X, G, U, act=ACT[name]), y, ey * (1 + half) + half * np.abs(y), "y")
    if name == "relu":
        dy = np.where(np.abs(a) <= ea, 0.0, dy)
        DY = t(dy)
    got = sm.gated_grad(DY, X, G, U, act=ACT[name])
    s = L.slope(name, a)
    da, db = dy * b * s, dy * h
    eda = act_error(a, ea, np.abs(dy) * (np.abs(b) + eb)) + np.abs(dy * s) * eb + fine * np.abs(da)
    edb = act_error(a, ea, dy) + fine * np.abs(db)
    eda, edb = eda * (1 + half) + half * np.abs(da), edb * (1 + half) + half * np.abs(db)
    ma, mb = np.abs(da) + eda, np.abs(db) + edb
    aw, au, ax = np.abs(wg), np.abs(wu), np.abs(x)
    for q, want, e, mags, k in (
            (got[0], da @ wg + db @ wu, eda @ aw + edb @ au, ma @ aw + mb @ au, 2 * n),
            (got[1], da.T @ x, eda.T @ ax, ma.T @ ax, T), (got[2], db.T @ x, edb.T @ ax, mb.T @ ax, T)):
        e = e + sum_error(k, mags)
        close(q, want, e * (1 + half) + half * np.abs(want), "gradient")


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(gpu_lib, name):
    """A gradient along a direction is the difference of the loss there.  Central differences of
    the float64 oracle with step h err by h^2 (third derivatives of order 1 here: 1e-6 of the sum
    of magnitudes); the float32 gradients by less."""
    T, d, n, h = 6, 20, 14, 1e-3
    rng = np.random.default_rng(11)
    t = lambda v: torch.from_numpy(v).float().cuda()
    f = lambda *s: rng.standard_normal(s).astype(np.float32).astype(np.float64)
    x, wg, wu, dy, bias = f(T, d), f(n, d) / 4, f(n, d) / 4, f(T, n), f(n)
    bi = {"bias": t(bias)}

    def check(got, inputs, loss):
        for k, g in enumerate(got):
            for _ in range(5):
                v = rng.standard_normal(inputs[k].shape)
                at = lambda s: loss(*[q + s * v if i == k else q for i, q in enumerate(inputs)])
                diff = (at(h) - at(-h)) / (2 * h)
                mags = float(np.sum(np.abs(np64(g)) * np.abs(v)))
                assert abs(diff - float(np.sum(np64(g) * v))) <= 2e-5 * mags + 2e-5

    check(sm.gated_grad(t(dy), t(x), t(wg), t(wu), act=ACT[name]), (x, wg, wu),
          lambda x, wg, wu: float(np.sum(dy * L.gated(x, wg, wu, name))))
    check(sm.linear_grad(t(dy), t(x), t(wg), act=ACT[name], **bi), (x, wg, bias),
          lambda x, w, b: float(np.sum(dy * L.linear(x, w, b, name))))


@pytest.mark.parametrize("name", L.ACTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_activations_over_their_whole_range(gpu_lib, dt, name):
    """Through a 1 x 1 weight of 1, so that z is x.  An exponent's argument (z, z^2 / 2, 2u) is off
    by a few 2^-24 of it, and the value by as much times itself: 2^-20 (1 + argument) of the value
    covers that, down to where e^-arg leaves float32's range (1 / (1 + e^88) is 6e-39 or 0, times
    |z| <= 15 there: 1e-37, and |z| times that in h); a slope by 2^-19 (1 + |z|) (up to 20, where it no longer changes) of 1.  Finite z
    give finite results, however large."""
    z = np.concatenate([np.linspace(-30, 30, 6001), [0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 1e10, -1e10,
                                                     1e19, -1e19, 1e30, -1e30, 3e38, -3e38]])
    x = torch.from_numpy(z).to(DT[dt]).cuda()[:, None]
    z = np64(x)[:, 0]
    w = torch.ones(1, 1, dtype=DT[dt], device="cuda")
    with np.errstate(over="ignore"):
        cut = np.clip(z, -1e4, 1e4)   # the oracle's own cubes stay finite
        want = np.where(np.abs(z) <= 1e4, L.act(name, cut), z if name == "none" else np.maximum(z, 0))
        arg = {"gelu": cut ** 2, "gelu_tanh": 1.6 * np.abs(cut + 0.044715 * cut ** 3)}.get(name, np.abs(cut))
    half = HALF[dt]
    got = np64(sm.linear(x, w, act=ACT[name]))[:, 0]
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= (2.0 ** -20 * (1 + np.minimum(arg, 200)) + half) * np.abs(want) + 1e-37)
    dx, _, db = sm.linear_grad(torch.ones_like(x), x, w, bias=torch.zeros(1, dtype=DT[dt], device="cuda"),
                               act=ACT[name], need_dw=False)
    slope = np64(dx)[:, 0]
    want = L.slope(name, cut)
    assert np.isfinite(slope).all()
    assert np.all(np.abs(slope - want) <= 2.0 ** -19 * (1 + np.minimum(np.abs(z), 20)) + 2 * half * np.abs(want))
    h = np64(sm.gated(x, w, torch.ones_like(w), act=ACT[name]))[:, 0]   # act(z) z
    ok = np.abs(z) <= 1e4
    want = L.act(name, cut) * cut
    assert np.all((np.abs(h - want) <= (2.0 ** -19 * (1 + np.minimum(arg, 200)) + half) * np.abs(want)
                   + 1e-37 * (1 + np.abs(z)))[ok])
    x = torch.full_like(x[:1], float("nan"))
    assert sm.linear(x, w, act=ACT[name]).isnan().all()
    assert sm.linear_grad(torch.ones_like(x), x, w, act=ACT[name], need_dw=False)[0].isnan().all() or name == "none"


# ---------------------------------------------------------------- 8-bit checkpoints

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 8), (1, 31), (2, 32), (5, 33), (7, 100), (64, 256), (3, 1283)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_act8(gpu_lib, dt, T, d, layout):
    rng = np.random.default_rng(T + d)
    v = rng.standard_normal((T, d)) * np.exp(4 * rng.standard_normal((T, d)))
    v[rng.random((T, d)) < 0.1] = 0.0
    v[:, d // 2] = np.where(rng.random(T) < 0.5, 448.0, 1e-36)
    X = Guarded(v, dt, *layout)
    x = np64(X.t)
    kept = sm.act8_pack(X.t)
    codes, scales = L.act8_pack(x)
    np.testing.assert_array_equal(kept.scale.view(torch.uint8).cpu().numpy(), scales)
    np.testing.assert_array_equal(kept.codes.view(torch.uint8).cpu().numpy(), codes)
    for to in ("f32", "bf16"):
        out = Guarded(np.full((T, d), np.nan), to, *layout)
        sm.act8_unpack(kept, DT[to], out=out.t)
        np.testing.assert_array_equal(np64(out.t), L.act8_unpack(codes, scales))
        out.check("values")
    # the values are their own checkpoint
    again = sm.act8_pack(sm.act8_unpack(kept, DT[dt]))
    assert torch.equal(sm.act8_unpack(again, torch.float32), sm.act8_unpack(kept, torch.float32))


def test_act8_extremes(gpu_lib):
    inf, nan = float("inf"), float("nan")
    rows = [[0.0] * 32, [-0.0] * 32, [inf] + [1.0] * 31, [nan, -inf] + [-3.0] * 30, [nan] * 32,
            [3.3e38] + [1.0] * 31, [1e-38] * 32, [2.0 ** -149] * 32, [2.0 ** -126] * 32,
            [2.0 ** -127] * 32, [448.0 * 2.0 ** -117] + [2.0 ** -126] * 31, [449.0] + [0.5] * 31]
    x = np.array(rows, np.float32)
    kept = sm.act8_pack(torch.from_numpy(x).cuda())
    codes, scales = L.act8_pack(x.astype(np.float64))
    np.testing.assert_array_equal(kept.scale.view(torch.uint8).cpu().numpy(), scales)
    np.testing.assert_array_equal(kept.codes.view(torch.uint8).cpu().numpy(), codes)
    for dt in DT.values():
        np.testing.assert_array_equal(np64(sm.act8_unpack(kept, dt)), L.act8_unpack(codes, scales))


def test_act8_every_code_and_scale(gpu_lib):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    got = sm.act8_unpack(sm.Act8(codes.cuda().view(torch.float8_e4m3fn),
                                 scales.cuda().view(torch.float8_e8m0fnu)), torch.float32)
    want = (codes.view(torch.float8_e4m3fn).double()
            * scales.view(torch.float8_e8m0fnu).double().repeat_interleave(32, 1)).float()
    np.testing.assert_array_equal(np64(got), want.double().numpy())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", [(1, 40, 24), (19, 33, 70), (140, 96, 200)])
def test_gradients_from_a_checkpoint_are_those_of_its_values(gpu_lib, dt, T, d, n):
    gen = torch.Generator().manual_seed(T)
    t = lambda *s: torch.randn(*s, generator=gen).to(DT[dt]).cuda()
    x, wg, wu, dy, bias = t(T, d), t(n, d), t(n, d), t(T, n), t(n)
    kept = sm.act8_pack(x)
    values = sm.act8_unpack(kept, DT[dt])
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))
    assert same(sm.gated_grad(dy, kept, wg, wu), sm.gated_grad(dy, values, wg, wu))
    for act in (sm.ACT_NONE, sm.ACT_GELU):
        assert same(sm.linear_grad(dy, kept, wg, bias=bias, act=act),
                    sm.linear_grad(dy, values, wg, bias=bias, act=act))


# ---------------------------------------------------------------- what may go wrong

@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_values_that_are_not_finite_stay_in_their_rows(gpu_lib, dt):
    T, d, n = 70, 40, 72
    gen = torch.Generator().manual_seed(5)
    t = lambda *s: torch.randn(*s, generator=gen).to(DT[dt]).cuda()
    x, wg, wu, dy = t(T, d), t(n, d), t(n, d), t(T, n)
    want, want_y = sm.gated_grad(dy, x, wg, wu, need_dw=False)[0], sm.gated(x, wg, wu)
    want_l = sm.linear(x, wg, act=sm.ACT_RELU)
    bad = x.clone()
    bad[T - 1, d - 1], bad[3, 0], bad[40] = float("nan"), float("inf"), float("nan")
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[T - 1, 3, 40]] = False
    y = sm.gated(bad, wg, wu)
    assert torch.equal(y[rows], want_y[rows])
    assert not y[[T - 1, 40]].isfinite().any()
    y = sm.linear(bad, wg, act=sm.ACT_RELU)
    assert torch.equal(y[rows], want_l[rows]) and y[[T - 1, 40]].isnan().all()
    dx = sm.gated_grad(dy, bad, wg, wu, need_dw=False)[0]
    assert torch.equal(dx[rows], want[rows]) and dx[[T - 1, 40]].isnan().all()
    # a NaN in dy reaches its row of dx and all of dw's rows that it enters
    bad = dy.clone()
    bad[2, 7] = float("nan")
    dx, dw, _ = sm.linear_grad(bad, x, wg)
    assert dx[2].isnan().all() and dx[3:].isfinite().all() and dx[:2].isfinite().all()
    assert dw[7].isnan().all() and dw[:7].isfinite().all() and dw[8:].isfinite().all()


def test_no_tokens(gpu_lib):
    w = torch.randn(24, 16, device="cuda")
    x, dy = torch.empty(0, 16, device="cuda"), torch.empty(0, 24, device="cuda")
    assert sm.linear(x, w).shape == (0, 24) and sm.gated(x, w, w).shape == (0, 24)
    dw, db = torch.full_like(w, 7.0), torch.full((24,), 7.0, device="cuda")
    sm.linear_grad(dy, x, w, bias=db.clone(), dw=dw, db=db, accumulate=True)
    assert bool((dw == 7).all()) and bool((db == 7).all())
    dx, dw, db = sm.linear_grad(dy, x, w, bias=db.clone(), dw=dw, db=db)
    assert dx.shape == (0, 16) and bool((dw == 0).all()) and bool((db == 0).all())
    dx, dwg, dwu = sm.gated_grad(dy, sm.act8_pack(x), w, w)
    assert bool((dwg == 0).all()) and bool((dwu == 0).all())
    assert sm.act8_unpack(sm.act8_pack(x), torch.float32).shape == (0, 16)


def test_leading_dimensions_and_slices(gpu_lib):
    gen = torch.Generator().manual_seed(9)
    wide = torch.randn(3, 5, 3 * 16, generator=gen).bfloat16().cuda()
    x = wide[..., 16:32]
    w = torch.randn(24, 2 * 16, generator=gen).bfloat16().cuda()
    flat = x.reshape(15, 16).contiguous()
    y = sm.gated(x, w[:, :16], w[:, 16:])
    assert y.shape == (3, 5, 24)
    assert torch.equal(y.view(15, 24), sm.gated(flat, w[:, :16].contiguous(), w[:, 16:].contiguous()))
    dy = torch.randn(3, 5, 24, generator=gen).bfloat16().cuda()
    dw = torch.zeros_like(w)     # both gradients side by side, as the weights
    before = wide.clone()
    sm.gated_grad(dy, x, w[:, :16], w[:, 16:], dx=wide[..., 32:], dwg=dw[:, :16], dwu=dw[:, 16:])
    want = sm.gated_grad(dy.view(15, 24), flat, w[:, :16].contiguous(), w[:, 16:].contiguous())
    assert torch.equal(wide[..., 32:].reshape(15, 16), want[0])
    assert torch.equal(wide[..., :32], before[..., :32])
    assert torch.equal(dw, torch.cat(want[1:], 1))


def test_front_end_refusals(gpu_lib):
    x, w, dy = (torch.randn(*s, device="cuda") for s in ((6, 16), (24, 16), (6, 24)))
    bad = [lambda: sm.linear(x.bfloat16(), w), lambda: sm.linear(x[:, :8], w),
           lambda: sm.linear(x, w, bias=torch.zeros(23, device="cuda")),
           lambda: sm.linear(x, w, residual=torch.zeros(5, 24, device="cuda")),
           lambda: sm.linear(x, w, out=torch.zeros(6, 23, device="cuda")),
           lambda: sm.linear(x, w.t().contiguous().t()), lambda: sm.linear(x, w, bias=w[:, 0]),
           lambda: sm.gated(x, w, w[:23]), lambda: sm.gated(x, w, w.bfloat16()),
           lambda: sm.linear(x, w.cpu()), lambda: sm.linear(x.cpu(), w),
           lambda: sm.linear_grad(dy[:5], x, w), lambda: sm.linear_grad(dy, sm.act8_pack(x[:5]), w),
           lambda: sm.linear_grad(dy, sm.act8_pack(x[:, :8].contiguous()), w),
           lambda: sm.linear_grad(dy, x, w, accumulate=True),
           lambda: sm.linear_grad(dy, x, w, dw=torch.zeros(24, 15, device="cuda")),
           lambda: sm.linear_grad(dy, x, w, ws=torch.zeros(8, dtype=torch.uint8)),
           lambda: sm.gated_grad(dy, x, w, w, dwg=w, accumulate=True),
           lambda: sm.linear_grad(dy, sm.Act8(x, x), w)]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: sm.linear(x, w, act=9), lambda: sm.linear_grad(dy, x, w, dw=w),
                 lambda: sm.linear(x[:1].expand(6, 16), w),
                 lambda: sm.linear(x.expand(2, 6, 16)[:, 0], w),
                 lambda: sm.linear_grad(dy, x, w, need_dx=False, need_dw=False)):
        with pytest.raises(sm.SmError):
            call()


def test_on_another_stream_and_in_a_graph(gpu_lib):
    gen = torch.Generator().manual_seed(2)
    t = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    T, d, n = 150, 136, 264
    x, wg, wu, wd, bias, dy = t(T, d), t(n, d), t(n, d), t(d, n), t(d), t(T, d)
    static = {}

    def work():
        kept = sm.act8_pack(x)
        h = sm.gated(x, wg, wu)
        kept_h = sm.act8_pack(h)
        y = sm.linear(h, wd, bias=bias, residual=x)
        dh, dwd, db = sm.linear_grad(dy, kept_h, wd, bias=bias)
        dx, dwg, dwu = sm.gated_grad(dh, kept, wg, wu)
        return [y, dx, dwg, dwu, dwd, db]

    want = [v.clone() for v in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = work()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        static["out"] = work()
    for k in range(4):      # eager work and new inputs between the replays
        x.copy_(t(T, d))
        dy.copy_(t(T, d))
        want = [v.clone() for v in work()]
        for v in static["out"]:
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(static["out"], want)), k
    del g
    gc.collect()


def test_the_same_call_gives_the_same_bits(gpu_lib):
    gen = torch.Generator().manual_seed(4)
    t = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    for T, d, n in ((2, 520, 300), (300, 264, 520), (1000, 128, 192)):
        x, wg, wu, dy, b = t(T, d), t(n, d), t(n, d), t(T, n), t(n)
        first = [*sm.gated_grad(dy, x, wg, wu), sm.gated(x, wg, wu),
                 *sm.linear_grad(dy, x, wg, bias=b, act=sm.ACT_GELU)]
        for _ in range(3):
            again = [*sm.gated_grad(dy, x, wg, wu), sm.gated(x, wg, wu),
                     *sm.linear_grad(dy, x, wg, bias=b, act=sm.ACT_GELU)]
            assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_two_streams_at_once_and_graphs_that_share_a_workspace(gpu_lib):
    gen = torch.Generator().manual_seed(12)
    t = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    T, d, n = 300, 520, 264          # products with split sums: all scratch is in use
    a = [t(T, n), t(T, d), t(n, d), t(n, d)]
    b = [t(T, n), t(T, d), t(n, d), t(n, d)]
    want = [[v.clone() for v in sm.gated_grad(*q)] for q in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, q in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(sm.gated_grad(*q))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, w in zip(got, want) for p, q in zip(g, w))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for q in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sm.gated_grad(*q, ws=ws))
        graphs.append(g)
    for _ in range(3):               # one after the other on one stream
        for g in graphs:
            g.replay()
        ws.fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, w in zip(outs, want) for p, q in zip(g, w))


def test_a_workspace_too_small_for_the_call(gpu_lib):
    x, w, dy = (torch.randn(*s, device="cuda") for s in ((300, 520), (264, 520), (300, 264)))
    with pytest.raises(ValueError, match="workspace too small"):
        sm.gated_grad(dy, x, w, w, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))


def test_offsets_beyond_32_bits(gpu_lib):
    """An input of 4.6 GB: its last rows, read along k and across it, and its checkpoint."""
    T, d, n = 70001, 32776, 24
    gen = torch.Generator(device="cuda").manual_seed(3)
    f = lambda top, *s: torch.randint(-top, top + 1, s, generator=gen, device="cuda",
                                      dtype=torch.int8).bfloat16()
    x, w, dy = f(1, T, d), f(1, n, d), f(1, T, n)
    y = sm.linear(x, w)
    dx, dw, _ = sm.linear_grad(dy, x, w)
    kept = sm.act8_pack(x)
    dw8 = sm.linear_grad(dy, kept, w, need_dx=False)[1]
    assert torch.equal(dw8, dw)      # whole numbers up to 1 are exact in 8 bits
    del dw8
    sums = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    W = w.double()
    for r in range(0, T, 10000):
        X, D = x[r:r + 10000].double(), dy[r:r + 10000].double()
        assert torch.equal(y[r:r + 10000], (X @ W.T).bfloat16())
        assert torch.equal(dx[r:r + 10000], (D @ W).bfloat16())
        sums += D.T @ X
    assert torch.equal(dw, sums.bfloat16())
    del dx, X, D
    assert torch.equal(sm.act8_unpack(kept, torch.bfloat16), x)


def test_rows_far_apart(gpu_lib):
    """Rows 32 MB apart (laid out before they are multiplied), results as well."""
    T, d, n, ld = 40, 24, 40, 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(6)
    f = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda").bfloat16()
    wide = torch.zeros(T, ld, dtype=torch.bfloat16, device="cuda")
    x, out, dx = wide[:, :d], wide[:, 100:100 + n], wide[:, 5000:5000 + d]
    x.copy_(f(T, d))
    w, dy = f(n, d), f(T, n)
    sm.linear(x, w, out=out)
    assert torch.equal(out.double(), (x.double() @ w.double().T).bfloat16().double())
    _, dw, _ = sm.linear_grad(dy, x, w, dx=dx)
    assert torch.equal(dx.double(), (dy.double() @ w.double()).bfloat16().double())
    assert torch.equal(dw.double(), (dy.double().T @ x.double()).bfloat16().double())


# ---------------------------------------------------------------- together

def test_a_training_step_of_a_gated_block(gpu_lib):
    """Two workers' batches through a block with 8-bit checkpoints, their gradients into the
    streams of a Sign-Muon step and of an AdamW step: as from the oracle's gradients."""
    M, T, d, n = 2, 40, 64, 96
    rng = np.random.default_rng(8)
    f = lambda *s, size=1.0: torch.from_numpy(size * rng.standard_normal(s)).float().cuda()
    wg, wu, wd = f(n, d, size=0.1), f(n, d, size=0.1), f(d, n, size=0.1)
    bias = torch.zeros(d, device="cuda")
    mats = [sm.MatrixBuffers(w=w, mom=torch.zeros(M, *w.shape, device="cuda"),
                             grad=torch.empty(M, *w.shape, device="cuda")) for w in (wg, wu, wd)]
    gb = torch.empty(M, d, device="cuda")
    rest = sm.ParamSet([sm.ParamBuffers.with_state(bias, gb)], M=M)
    want = []
    for k in range(M):
        x, dy = f(T, d), f(T, d)
        kept = sm.act8_pack(x)
        h = sm.gated(x, wg, wu)
        kept_h = sm.act8_pack(h)
        y = sm.linear(h, wd, bias=bias, residual=x)
        np.testing.assert_allclose(np64(y), L.linear(L.gated(np64(x), np64(wg), np64(wu)), np64(wd))
                                   + np64(x), atol=2e-5)
        dh, _, _ = sm.linear_grad(dy, kept_h, wd, bias=bias, dw=mats[2].grad[k], db=gb[k])
        sm.gated_grad(dh, kept, wg, wu, dwg=mats[0].grad[k], dwu=mats[1].grad[k], need_dx=False)
        xv, hv = (np64(sm.act8_unpack(q, torch.float32)) for q in (kept, kept_h))
        wdh, wdw, wdb = L.linear_grad(np64(dy), hv, np64(wd))
        _, wgg, wgu = L.gated_grad(wdh, xv, np64(wg), np64(wu))
        want.append((wgg, wgu, wdw, wdb))
    # sums of up to 100 products of order one in float32: 1e-4 covers them
    for i, mb in enumerate(mats):
        np.testing.assert_allclose(np64(mb.grad), np.stack([g[i] for g in want]), atol=1e-4)
    np.testing.assert_allclose(np64(gb), np.stack([g[3] for g in want]), atol=1e-4)
    before = [w.clone() for w in (wg, wu, wd, bias)]
    muon = sm.ParamSet([sm.ParamBuffers(grad=mb.grad) for mb in mats], M=M)
    clip = sm.grad_norm([muon, rest], max_norm=1.0)
    total = np.sqrt(sum(np.sum(np.mean([g[i] for g in want], 0) ** 2) for i in range(4)))
    assert abs(float(clip[0]) - total) <= 1e-5 * total
    sm.step(sm.StepConfig(algo=sm.SIGN_MUON, M=M, lr=1e-3), mats, 1)
    sm.adamw(sm.AdamWConfig(lr=1e-3), rest, 1, gscale=clip[1:])
    for a, b in zip(before, (wg, wu, wd, bias)):
        moved = (a - b).abs()
        assert bool((moved <= 1.01e-3).all()) and float(moved.max()) >= 0.99e-3
    rest.close()
    muon.close()
