"""The curved activations of the feed-forward layers in every way that a product
is launched (tiles of 256, 128 and 64, columns cut off for a second launch, sums
in shares), on the GPU against references in float64.
tests/test_layer_plan_cpu.py holds SHAPES to their purpose.

Bounds: those of tests/test_gpu_layer.py.  A float32 sum of K products is off
by at most K * 2^-23 of the sum of the products' magnitudes; an activation or
its slope by 1.13 times that and 2^-20 (1 + |z|) for its own evaluation; a
result, and dz ahead of the sums that it enters, by half a step of its type.
"""
import math

import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm
from tests.test_gpu_layer import ACT, DT, HALF

pytestmark = pytest.mark.gpu

# (T, d, n)
SHAPES = [(1003, 1280, 3416), (4200, 72, 4104), (4090, 72, 4091), (2051, 260, 2053),
          (200, 4101, 1003), (150, 2000, 300), (1200, 40, 1300)]
CURVED = ["silu", "gelu", "gelu_tanh"]


def both64(name, z):
    """act(z) and act'(z) of float64 z."""
    if name == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u, du = z, 1.0
    if name == "gelu_tanh":   # (1 + tanh(u / 2)) / 2 is the logistic function of u
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(u)
    return z * p, p + z * p * torch.sigmoid(-u) * du


def sum_error(K, mags):
    return K * 2.0 ** -23 * mags


def act_error(z, ez, scale):
    return scale.abs() * (1.13 * ez + 2.0 ** -20 * (1 + z.abs()))


def close(got, want, error, half, what):
    """error: before the result's own rounding."""
    off = (got.double() - want).abs()
    bound = error * (1 + half) + half * want.abs()
    worst = float((off / bound).max())
    assert bool((off <= bound).all()), f"{what}: {worst:.2f} times its bound"


def inputs(seed, dt, *shapes):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(size * torch.randn(*s, generator=gen, device="cuda")).to(DT[dt]) for size, s in shapes]


@pytest.mark.parametrize("name", CURVED)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_curved_activations_linear(gpu_lib, T, d, n, dt, name):
    half, size = HALF[dt], d ** -0.5
    x, w, bias, res, dy, old, old_b = inputs(T + d, dt, (1, (T, d)), (3 * size, (n, d)), (1, (n,)),
                                             (1, (T, n)), (1, (T, n)), (1, (n, d)), (1, (n,)))
    X, W, BI, R, DY = (v.double() for v in (x, w, bias, res, dy))
    z = X @ W.T + BI
    ez = sum_error(d + 1, X.abs() @ W.abs().T + BI.abs())
    a, slope = both64(name, z)
    y = a + R
    one = torch.ones_like(z)
    close(sm.linear(x, w, bias=bias, act=ACT[name], residual=res), y,
          act_error(z, ez, one) + 2.0 ** -23 * (y.abs() + R.abs()), half, "y")
    dz = DY * slope
    e = act_error(z, ez, DY)
    e = e * (1 + half) + half * dz.abs()
    m = dz.abs() + e
    dw, db = old.clone(), old_b.clone()
    dx, _, _ = sm.linear_grad(dy, x, w, bias=bias, act=ACT[name], dw=dw, db=db, accumulate=True)
    close(dx, dz @ W, e @ W.abs() + sum_error(n, m @ W.abs()), half, "dx")
    for got, before, want, err, mags in ((dw, old, dz.T @ X, e.T @ X.abs(), m.T @ X.abs()),
                                         (db, old_b, dz.sum(0), e.sum(0), m.sum(0))):
        before = before.double()
        close(got, want + before, err + sum_error(T + 1, mags + before.abs()), half, "dw, db")


@pytest.mark.parametrize("name", CURVED)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_curved_activations_gated(gpu_lib, T, d, n, dt, name):
    half, size, fine = HALF[dt], d ** -0.5, 2.0 ** -22   # fine: the epilogue's products
    x, wg, wu, dy = inputs(T + d + 1, dt, (1, (T, d)), (3 * size, (n, d)), (size, (n, d)), (1, (T, n)))
    X, G, U, DY = (v.double() for v in (x, wg, wu, dy))
    a, b = X @ G.T, X @ U.T
    ea, eb = (sum_error(d, X.abs() @ v.abs().T) for v in (G, U))
    h, slope = both64(name, a)
    close(sm.gated(x, wg, wu, act=ACT[name]), h * b,
          act_error(a, ea, b.abs() + eb) + h.abs() * eb + fine * (h * b).abs(), half, "y")
    da, db = DY * b * slope, DY * h
    eda = act_error(a, ea, DY.abs() * (b.abs() + eb)) + (DY * slope).abs() * eb + fine * da.abs()
    edb = act_error(a, ea, DY) + fine * db.abs()
    eda, edb = eda * (1 + half) + half * da.abs(), edb * (1 + half) + half * db.abs()
    ma, mb = da.abs() + eda, db.abs() + edb
    g, u, ax = G.abs(), U.abs(), X.abs()
    dx, dwg, dwu = sm.gated_grad(dy, x, wg, wu, act=ACT[name])
    close(dx, da @ G + db @ U, eda @ g + edb @ u + sum_error(2 * n, ma @ g + mb @ u), half, "dx")
    close(dwg, da.T @ X, eda.T @ ax + sum_error(T, ma.T @ ax), half, "dwg")
    close(dwu, db.T @ X, edb.T @ ax + sum_error(T, mb.T @ ax), half, "dwu")


# both kernels that few tokens may take: narrow outputs of long sums, wide ones, odd ones
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("gap", [0, 5, 8])
@pytest.mark.parametrize("d,n", [(11008, 512), (2304, 768), (4096, 64), (4100, 1003), (264, 4096)])
def test_few_tokens(gpu_lib, d, n, gap, dt):
    """Whole numbers: every sum is exact, whichever kernel takes it and however it is split."""
    gen = torch.Generator(device="cuda").manual_seed(d + n + gap)

    def whole(top, *s):
        wide = torch.randint(-top, top + 1, (*s[:-1], s[-1] + gap), generator=gen, device="cuda")
        return wide.to(DT[dt])[..., :s[-1]]

    wg, wu, bias = whole(2, n, d), whole(1, n, d), whole(9, n).contiguous()
    G, U, BI = (v.double() for v in (wg, wu, bias))
    for T in (1, 2, 8, 15, 16, 17, 24, 31, 32, 33):
        x, res = whole(1, T, d), whole(20, T, n)
        X = x.double()
        a, b = X @ G.T, X @ U.T
        wide = torch.full((T + 2, n + gap), float("nan"), device="cuda", dtype=DT[dt])
        out = wide[1:T + 1, :n]
        sm.linear(x, wg, bias=bias, act=sm.ACT_RELU, residual=res, out=out)
        assert torch.equal(out, ((a + BI).relu() + res.double()).to(DT[dt]))
        sm.gated(x, wg, wu, act=sm.ACT_RELU, out=out)
        assert torch.equal(out, (a.relu() * b).to(DT[dt]))
        out.fill_(float("nan"))
        assert bool(wide.isnan().all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,n", [(11008, 512), (4096, 11008)])
def test_few_tokens_that_are_laid_out(gpu_lib, d, n, dt):
    """x off alignment beside weights that are read in place; scratch full of NaN, of the size asked
    for; the same bits again, and from a graph."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    whole = lambda top, *s: torch.randint(-top, top + 1, s, generator=gen, device="cuda").to(DT[dt])
    wg, wu = whole(2, n, d), whole(1, n, d)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for T in (1, 19, 32):
        x = whole(1, T, d + 3)[:, 3:]
        want = ((x.double() @ wg.double().T).relu() * (x.double() @ wu.double().T)).to(DT[dt])
        first = sm.gated(x, wg, wu, act=sm.ACT_RELU, ws=ws)
        assert torch.equal(first, want)
        assert torch.equal(sm.linear(x, wu, ws=ws), (x.double() @ wu.double().T).to(DT[dt]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sm.gated(x, wg, wu, act=sm.ACT_RELU)
        for _ in range(3):
            out.fill_(float("nan"))
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        del g
