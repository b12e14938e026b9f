"""Calls of the feed-forward layers that leave gradients out, workspaces over
tensors, and values that are not finite, on the GPU.

Gradients left out: against the same call with all of them.  Bit for bit, but for the two weight gradients
of a gated layer: they are one launch if both are wanted, whose sums may be
split otherwise than one's.  Two float32 sums of T products (and an addend) in
another order are apart by twice (T + 1) * 2^-23 of the magnitudes' sum, and
their roundings by twice half a step."""
import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm

pytestmark = pytest.mark.gpu


def tensors(seed, dtype, *shapes):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=gen).to(dtype).cuda() for s in shapes]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", [sm.ACT_NONE, sm.ACT_GELU])
@pytest.mark.parametrize("T,d,n", [(3, 17, 40), (300, 136, 72)])
def test_a_frozen_bias(gpu_lib, T, d, n, act, dtype):
    x, w, bias, dy, old = tensors(1, dtype, (T, d), (n, d), (n,), (T, n), (n, d))
    want = sm.linear_grad(dy, x, w, bias=bias, act=act)
    got = sm.linear_grad(dy, x, w, bias=bias, act=act, need_db=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] is None
    # added to a stream, with no gradient of the bias to add to
    dw, both = old.clone(), old.clone()
    got = sm.linear_grad(dy, x, w, bias=bias, act=act, dw=dw, need_db=False, accumulate=True)
    sm.linear_grad(dy, x, w, bias=bias, act=act, dw=both, db=bias.clone(), accumulate=True)
    assert got[1] is dw and got[2] is None and torch.equal(dw, both)
    # a gradient that is given and not wanted stays as it is
    db = bias.clone()
    assert sm.linear_grad(dy, x, w, bias=bias, act=act, db=db, need_db=False)[2] is None
    assert torch.equal(db, bias)
    with pytest.raises(ValueError, match="accumulate needs db"):
        sm.linear_grad(dy, x, w, bias=bias, act=act, dw=dw, accumulate=True)
    with pytest.raises(sm.SmError):   # nothing is wanted
        sm.linear_grad(dy, x, w, bias=bias, act=act, need_dx=False, need_dw=False, need_db=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,n", [(3, 17, 40), (300, 136, 72)])
def test_one_frozen_projection(gpu_lib, T, d, n, dtype):
    x, wg, wu, dy, old = tensors(2, dtype, (T, d), (n, d), (n, d), (T, n), (n, d))
    streams = [old.clone(), old.clone()]
    sm.gated_grad(dy, x, wg, wu, dwg=streams[0], dwu=streams[1], accumulate=True)
    want = sm.gated_grad(dy, x, wg, wu)
    half = torch.finfo(dtype).eps / 2
    X, G, U, DY = (v.double() for v in (x, wg, wu, dy))
    # silu's slope is at most 1.1, and |silu(a)| at most |a|
    mags = [(1.1 * (DY * (X @ v.T)).abs()).T @ X.abs() * (1 + half) for v in (U, G)]

    def near(got, full, k, added=0.0):
        sums = (T + 1) * 2.0 ** -23 * (mags[k] + added)
        bound = 2 * ((1 + half) * sums + half * full.double().abs() * (1 + 2 * half))
        assert bool(((got.double() - full.double()).abs() <= bound).all())

    for k, names in enumerate((("need_dwu", "dwg"), ("need_dwg", "dwu"))):
        got = sm.gated_grad(dy, x, wg, wu, **{names[0]: False})
        assert torch.equal(got[0], want[0]) and got[2 - k] is None
        near(got[1 + k], want[1 + k], k)
        new = old.clone()
        got = sm.gated_grad(dy, x, wg, wu, **{names[0]: False, names[1]: new}, accumulate=True)
        assert got[1 + k] is new
        near(new, streams[k], k, old.double().abs())
        with pytest.raises(ValueError, match="accumulate needs"):
            sm.gated_grad(dy, x, wg, wu, **{names[0]: False}, accumulate=True)


def test_a_workspace_over_a_tensor_is_refused(gpu_lib):
    x, w, dy = tensors(3, torch.float32, (300, 520), (264, 520), (300, 264))
    flat = torch.zeros(64 << 18, device="cuda")
    out = flat[4096:4096 + 300 * 264].view(300, 264)
    before = x.clone()
    with pytest.raises(sm.SmError):
        sm.linear(x, w, out=out, ws=flat)
    with pytest.raises(sm.SmError):
        sm.gated_grad(out, x, w, w, ws=flat)
    assert bool((flat == 0).all()) and torch.equal(x, before)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", [sm.ACT_NONE, sm.ACT_RELU, sm.ACT_SILU, sm.ACT_GELU, sm.ACT_GELU_TANH])
@pytest.mark.parametrize("T,d,n", [(20, 264, 520), (300, 1000, 264), (2051, 260, 2053), (4090, 72, 4091)])
def test_values_that_are_not_finite_reach_their_rows_alone(gpu_lib, T, d, n, act, dtype):
    """In every way that the products are launched; the other rows keep their bits."""
    x, wg, wu, dy, res = tensors(4, dtype, (T, d), (n, d), (n, d), (T, n), (T, n))
    wg[0], wg[1], wu[0] = 0.0, -wg[2], 0.0
    bad_x, bad_dy = x.clone(), dy.clone()
    bad_x[T - 1, d - 1], bad_x[3, 0], bad_x[7, 5] = float("nan"), float("inf"), -float("inf")
    bad_dy[T // 2, n - 1], bad_dy[11, 1] = float("nan"), float("inf")
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[T - 1, 3, 7]] = False
    for call in (lambda x: sm.linear(x, wg, act=act, residual=res), lambda x: sm.gated(x, wg, wu, act=act)):
        got, want = call(bad_x), call(x)
        assert torch.equal(got[rows], want[rows]) and got[T - 1].isnan().all()
    if act == sm.ACT_RELU:   # infinity by the sign of its weight; times 0 it is NaN
        y = sm.linear(bad_x, wg, act=act)
        want = torch.where(wg[1:, 0] > 0, float("inf"), 0.0)
        assert torch.equal(y[3, 1:].float(), want) and y[3, 0].isnan()
    rows[[T // 2, 11]] = False
    for call in (lambda x, dy: sm.linear_grad(dy, x, wg, act=act, need_dw=False),
                 lambda x, dy: sm.gated_grad(dy, x, wg, wu, act=act, need_dw=False)):
        got, want = call(bad_x, bad_dy)[0], call(x, dy)[0]
        assert torch.equal(got[rows], want[rows])
        assert not got[T // 2].isfinite().any()
