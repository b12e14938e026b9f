"""AdamW over parameter sets, the global gradient norm and the 8-bit states
on the GPU, against the float64 oracle.

Tolerances.  A float32 value that the kernel computes from stored inputs by
k roundings is off by at most k * 2^-24 of its terms (half a step each):

* m: three roundings of each term (gradient's scaling, product, sum) and
  one of (1 - beta): 2^-21 * (|b1 m| + |(1-b1) g|) covers them twice over.
  v the same, with g twice: 2^-20.
* the step's change d: m and v as above, square root and reciprocal within
  one step each, six more products: 2^-19 * d, and the cancellation inside
  m: 2^-21 * lr/(1-b1^t) * terms / denominator.
* w: the change's bound, three roundings of w: 2^-22 |w|; then half a step of
  the type (bf16: 2^-8 of the value, for a stochastic rounding a whole one).

8-bit codes: the oracle rounds the interval that m may lie in; the code must
be between the two ends (in almost all cases they agree), and its block's
scale one that the interval of its largest entry allows.
"""
import gc
import weakref

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm
from matrix_aware_optimizer_momentum_amd import workloads as W
from oracle import adamw_oracle as A

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def np64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def raw(t):
    """The tensor's bytes."""
    return t.detach().contiguous().view(-1).view(torch.uint8).cpu().numpy()


class Case:
    """One parameter: buffers inside larger ones (sentinels around them)."""

    PAD = 64
    base = 0     # index of the first entry in its parameter

    def __init__(self, n, w="f32", g="f32", fp8=False, M=1, shift=0, wd=0.0, lr_mult=1.0,
                 gen=None, zero=False, gsize=1e-2, stride=None):
        self.n, self.w_kind, self.fp8, self.M, self.wd, self.lr_mult = n, w, fp8, M, wd, lr_mult
        gen = gen or np.random.default_rng(n)
        self.pads = []
        stride = stride or n

        def place(x, dtype=None):
            x = torch.as_tensor(np.asarray(x, np.float32)).to(dtype) if not torch.is_tensor(x) else x
            size = x.element_size()
            buf = torch.full(((2 * self.PAD + x.numel() + shift) * size,), 0xA5, dtype=torch.uint8,
                             device="cuda")
            a = (self.PAD + shift) * size
            if x.numel():
                buf[a:a + x.numel() * size] = x.reshape(-1).view(torch.uint8).cuda()
            self.pads.append((buf, a, a + x.numel() * size))
            return buf[a:a + x.numel() * size].view(x.dtype)

        size = gsize * np.exp(gen.standard_normal(max(1, -(-n // 256))).repeat(256)[:n])
        master = 0.02 * gen.standard_normal(n)
        wdt = DT["f32"] if w == "f32" else DT["bf16"]
        self.w = place(master, wdt)
        self.master = place(master, torch.float32) if w == "master" else None
        rows = np.zeros((M, stride), np.float32)
        rows[:, :n] = size * gen.standard_normal((M, n))
        grad = place(rows, DT[g])
        self.grad = torch.as_strided(grad, (M, n), (stride, 1))
        m0 = 0.0 if zero else 0.3 * size * gen.standard_normal(n)
        v0 = 0.0 if zero else (size * gen.standard_normal(n)) ** 2 + 0.1 * size * size
        m0, v0 = np.broadcast_to(m0, n).astype(np.float32), np.broadcast_to(v0, n).astype(np.float32)
        if fp8:
            parts = []
            for x, kind, dt in ((m0, "m", torch.float8_e4m3fn), (v0, "v", torch.float8_e5m2)):
                c, s = A.pack(x.astype(np.float64), kind) if n else (np.zeros(0), np.zeros(0))
                parts += [torch.from_numpy(c.astype(np.float32)).to(dt), s]
            self.m, self.v = place(parts[0]), place(parts[2])
            self.ms, self.vs = place(parts[1], torch.float32), place(parts[3], torch.float32)
        else:
            self.m, self.v = place(m0, torch.float32), place(v0, torch.float32)
            self.ms = self.vs = None

    def buffers(self):
        return sm.ParamBuffers(grad=self.grad, w=self.w, m=self.m, v=self.v, m_scale=self.ms,
                               v_scale=self.vs, master=self.master, weight_decay=self.wd,
                               lr_mult=self.lr_mult)

    def grad_only(self):
        return sm.ParamBuffers(grad=self.grad if self.M > 1 else self.grad[0])

    def grads64(self):
        return self.grad.double().cpu().numpy()

    def state64(self):
        m, v = np64(self.m.float()), np64(self.v.float())
        if self.fp8:
            m = m * A.per_entry(np64(self.ms), self.n)
            v = v * A.per_entry(np64(self.vs), self.n)
        return m, v

    def written(self):
        return [t for t in (self.w, self.m, self.v, self.ms, self.vs, self.master) if t is not None]

    def pads_intact(self):
        return all(bool((b[:a] == 0xA5).all()) and bool((b[e:] == 0xA5).all())
                   for b, a, e in self.pads)

    def expect(self, cfg, t, index, gscale=1.0, lr_scale=1.0):
        """What the step has to leave, from the buffers as they are now."""
        c = dict(lr=cfg.lr, beta1=cfg.beta1, beta2=cfg.beta2, eps=cfg.eps)
        m, v = self.state64()
        w = np64(self.w if self.master is None else self.master)
        grads = self.grads64()
        g, m1, v1 = A.moments(grads, m, v, c, gscale)
        b1, b2 = A.f32(cfg.beta1), A.f32(cfg.beta2)
        # ... and a denormal's step, but nothing where all terms are zero
        terms = np.abs(b1 * m) + np.abs((1 - b1) * g)
        m_off = 2.0 ** -21 * terms + np.where(terms > 0, 2.0 ** -149, 0.0)
        v_off = 2.0 ** -20 * v1 + np.where(v1 > 0, 2.0 ** -149, 0.0)
        w1, d = A.weights(w, m1, v1, t, c, self.wd, self.lr_mult, lr_scale)
        lr = cfg.lr * self.lr_mult * lr_scale
        den = np.sqrt(v1 / (1 - b2 ** t)) + cfg.eps
        w_off = 2.0 ** -19 * d + lr / (1 - b1 ** t) * m_off / den + 2.0 ** -22 * np.abs(w)
        return dict(cfg=cfg, t=t, index=index, m=m1, v=v1, w=w1, m_off=m_off, v_off=v_off,
                    w_off=w_off)

    def check(self, e, what=""):
        assert self.pads_intact(), what
        n = self.n
        if n == 0:
            return
        stochastic = e["cfg"].rounding == sm.ROUND_STOCHASTIC
        w = np64(self.w)
        half = 0.0
        if self.w_kind != "f32":
            half = 2.0 ** -8 * (np.abs(e["w"]) + e["w_off"]) * \
                (2 if stochastic and self.w_kind == "bf16" else 1)
        assert np.all(np.abs(w - e["w"]) <= e["w_off"] + half), (what, "w")
        if self.master is not None:
            master = np64(self.master)
            assert np.all(np.abs(master - e["w"]) <= e["w_off"]), (what, "master")
            assert torch.equal(self.w, self.master.to(torch.bfloat16)), (what, "rounding")
        elif stochastic and self.w_kind == "bf16":
            # the float32 value's neighbour that the random bits choose
            _, rw = A.random_bits(e["cfg"].seed, e["t"], e["index"], self.base + np.arange(n))
            ends = []
            for x in (e["w"] - e["w_off"], e["w"] + e["w_off"]):
                # magnitudes round away by the random bits: on each end's own magnitude
                a = np.abs(x)
                ex = np.frexp(a)[1] - 8
                q = np.ldexp(1.0, ex)
                ends.append(np.copysign(np.floor(a / q + rw.astype(float) / 65536) * q, x))
            assert np.all((w >= np.minimum(*ends)) & (w <= np.maximum(*ends))), (what, "w bits")
        if not self.fp8:
            m, v = np64(self.m), np64(self.v)
            assert np.all(np.abs(m - e["m"]) <= e["m_off"]), (what, "m")
            assert np.all(np.abs(v - e["v"]) <= e["v_off"]), (what, "v")
            return
        r, _ = A.random_bits(e["cfg"].seed, e["t"], e["index"], self.base + np.arange(n))
        for kind, x, off, code, scale, bits in (
                ("m", e["m"], e["m_off"], self.m, self.ms, r & np.uint64(0xFFFF)),
                ("v", e["v"], e["v_off"], self.v, self.vs, r >> np.uint64(16))):
            s = np64(scale)
            lo, hi = A.scales(np.maximum(np.abs(x) - off, 0), kind), A.scales(np.abs(x) + off, kind)
            assert np.all((s == lo) | (s == hi)), (what, kind, "scale")
            s = A.per_entry(s, n)
            got = np64(code.float())
            u = (bits.astype(float) + 0.5) / 65536
            ends = []
            for y in (np.abs(x) - off, np.abs(x) + off):
                q = A.to_grid(np.clip(y / s, 0, A.KINDS[kind][3]), kind, u)
                if kind == "v":
                    q = np.where(y > 0, np.maximum(q, 2.0 ** -16), q)
                ends.append(q)
            a = np.abs(got)
            assert np.all((a >= ends[0]) & (a <= ends[1])), (what, kind, "code")
            # nearly everywhere the code is determined
            assert np.mean(ends[0] != ends[1]) < 1e-2 or n < 1000, (what, kind)
            big = np.abs(x) > off
            assert np.all((np.sign(got) == np.sign(x))[big & (a > 0)]), (what, kind, "sign")


class Window(Case):
    """A parameter's entries from a on: n of them and the rest of the last one's
    block (the oracle takes a block's scale from all of its entries)."""

    def __init__(self, p, M, a, n):
        assert a % 256 == 0
        n = min(-(-n // 256) * 256, p.w.numel() - a)
        e, blocks = slice(a, a + n), slice(a // 256, -(-(a + n) // 256))
        self.n, self.M, self.base, self.pads = n, M, a, []
        self.wd, self.lr_mult, self.fp8 = p.weight_decay, p.lr_mult, p.m_scale is not None
        self.w_kind = "f32" if p.w.dtype == torch.float32 else \
            "bf16" if p.master is None else "master"
        self.w, self.m, self.v = p.w[e], p.m[e], p.v[e]
        self.grad = p.grad.view(M, -1)[:, e]
        self.ms, self.vs = (None, None) if not self.fp8 else (p.m_scale[blocks], p.v_scale[blocks])
        self.master = None if p.master is None else p.master[e]


def run_and_check(cases, M=1, t=5, gscale=None, steps=1, rounding=sm.ROUND_NEAREST, **cfg):
    cfg = sm.AdamWConfig(**{**dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, seed=0x1234567890AB,
                                   rounding=rounding), **cfg})
    pset = sm.ParamSet([c.buffers() for c in cases], M=M)
    gs = torch.tensor([gscale], device="cuda") if gscale is not None else None
    for k in range(steps):
        e = [c.expect(cfg, t + k, i, 1.0 if gscale is None else gscale)
             for i, c in enumerate(cases)]
        sm.adamw(cfg, pset, t + k, gscale=gs)
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            c.check(e[i], (i, c.n, t + k))
    return pset


# around the 8-bit states' blocks, a thread's, a wave's and a work item's share
LENGTHS = [511, 512, 513, 1023, 1025, 6143, 6144, 6145, 1, 2, 7, 8, 9, 63, 255, 256, 257, 2040, 2047, 2048, 2049, 4103, 20000, 0]


@pytest.mark.parametrize("w", ["f32", "bf16", "master"])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_step_over_many_lengths(gpu_lib, w, g, fp8):
    run_and_check([Case(n, w, g, fp8, wd=0.1 * (n % 2)) for n in LENGTHS], gscale=0.7, steps=2)


# Accesses are wide at any alignment: only a tensor's last entries, fewer than
# four, go one by one.
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_step_of_unaligned_buffers(gpu_lib, fp8):
    """Buffers at every element offset: the element-wise path."""
    run_and_check([Case(n, w, g, fp8, shift=sh, wd=0.05)
                   for n in (5, 300, 2100) for w, g in (("f32", "bf16"), ("master", "f32"),
                                                        ("bf16", "bf16")) for sh in (1, 3)])


# Odd rows take the same wide accesses as even ones.
@pytest.mark.parametrize("M", [2, 3, 64])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_step_on_the_mean_of_workers(gpu_lib, M, fp8):
    """Rows apart by a stride, even and odd ones (the odd bf16 rows take the
    element-wise path); entries between the rows are not read."""
    cases = [Case(n, "f32", g, fp8, M=M, stride=st) for n, st in
             ((300, 300), (301, 301), (301, 304), (2500, 4096)) for g in ("f32", "bf16")]
    run_and_check(cases, M=M, gscale=1.25)


def test_first_step_from_empty_states(gpu_lib):
    run_and_check([Case(700, "bf16", "bf16", f, zero=True) for f in (False, True)], t=1, steps=3)


def test_mixed_types_lr_mult_and_stochastic_weights(gpu_lib):
    cases = [Case(1000 + 37 * i, w, g, f, wd=0.1 * (i % 3), lr_mult=[1.0, 0.5, 0.0][i % 3])
             for i, (w, g, f) in enumerate((w, g, f) for w in ("f32", "bf16", "master")
                                           for g in ("f32", "bf16") for f in (False, True))]
    run_and_check(cases, rounding=sm.ROUND_STOCHASTIC, steps=2)


def test_many_parameters_take_several_table_launches(gpu_lib):
    run_and_check([Case(1 + (i * 7919) % 700, ["f32", "bf16"][i % 2], "f32", i % 3 == 0)
                   for i in range(150)])


def test_stochastic_states_follow_slow_averages(gpu_lib):
    """beta2 = 0.999 and a gradient a tenth of what built v: over 800 steps v
    falls to 0.999^800 = 0.449 of itself (+ the new 0.0055), where a rounding
    to nearest would never leave its code.  A step's rounding moves an entry
    by at most a quarter of v with probability 0.001 * 4: a relative variance
    of at most 800 * 0.25^2 * 0.004 = 0.2, for the mean of 4096 entries a
    deviation of 0.7 %; bound 4 % (5 sigma).  m has converged, and rounds with
    at most (2^-3 / 2)^2 a step, over 1 / (1 - 0.81) steps: 0.14, the mean
    0.22 %; bound 2 %."""
    n = 4096
    c = Case(n, "f32", "f32", True, zero=True)
    c.grad.fill_(0.1)
    m8, v8, ms, vs = sm.state8_pack(torch.zeros(n, device="cuda"), torch.ones(n, device="cuda"))
    for dst, src in ((c.m, m8), (c.v, v8)):
        dst.view(torch.uint8).copy_(src.view(torch.uint8))
    c.ms.copy_(ms)
    c.vs.copy_(vs)
    pset = sm.ParamSet([c.buffers()])
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(800):
        sm.adamw(sm.AdamWConfig(lr=0.0, beta2=0.999), pset, step=step)
    want = 0.999 ** 800 + 0.01 * (1 - 0.999 ** 800)
    _, v = c.state64()
    assert int(step) == 800
    assert abs(v.mean() / want - 1) < 0.04
    m, _ = c.state64()
    assert abs(m.mean() / 0.1 - 1) < 0.02


def test_entries_far_beyond_32_bits(gpu_lib):
    """2^32 + 2600 entries with 8-bit states: the far end's offsets, scales and
    random bits (bf16 weights, 26 GB in all)."""
    n = (1 << 32) + 2600
    dev = "cuda"
    w = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    p = sm.ParamBuffers.with_state(w, g, fp8=True)
    spots = [0, (1 << 31) - 512, (1 << 32) - 1024, (n - 1200) // 256 * 256]
    rng = np.random.default_rng(3)
    for a in spots:
        k = min(1536, n - a)
        g[a:a + k].copy_(torch.from_numpy(rng.standard_normal(k).astype(np.float32)))
    cfg = sm.AdamWConfig(lr=1e-2, beta1=0.9, beta2=0.99, seed=99)
    sm.adamw(cfg, sm.ParamSet([p]), 1)
    torch.cuda.synchronize()
    c = dict(lr=cfg.lr, beta1=cfg.beta1, beta2=cfg.beta2, eps=cfg.eps)
    for a in spots:
        k = min(1536, n - a)
        e = slice(a, a + k)
        gg = np64(g[e])[None]
        _, m, v = A.moments(gg, 0.0, 0.0, c)
        wv, _ = A.weights(0.0, m, v, 1, c)
        assert np.all(np.abs(np64(w[e]) - wv) <= 2.0 ** -8 * np.abs(wv) + 1e-7), a
        r, _ = A.random_bits(99, 1, 0, np.arange(a, a + k))
        for kind, x, code, scale, bits in (("m", m, p.m, p.m_scale, r & np.uint64(0xFFFF)),
                                           ("v", v, p.v, p.v_scale, r >> np.uint64(16))):
            s = A.scales(x, kind)
            assert np.array_equal(np64(scale[a // 256:a // 256 + len(s)]), s), (a, kind)
            want = np.sign(x) * A.to_grid(np.abs(x) / A.per_entry(s, k), kind,
                                          (bits.astype(float) + 0.5) / 65536)
            if kind == "v":
                want = np.where(x > 0, np.maximum(want, 2.0 ** -16), want)
            # a float32 value within 2^-20 of a threshold may fall either way
            assert np.mean(np64(code[e].float()) != want) < 5e-3, (a, kind)
    del w, g, p


# Runs of items per XCD are taken by sets of any size that have enough items.
@pytest.mark.parametrize("n,w,g,fp8,M", [
    (30_000_001, "bf16", "bf16", False, 1), (20_000_003, "f32", "f32", False, 1),
    (18_000_002, "f32", "f32", False, 2), (60_000_001, "bf16", "bf16", True, 1),
    (36_000_513, "master", "f32", True, 1), (40_000_004, "master", "bf16", True, 3),
])
def test_sets_beyond_the_cache(gpu_lib, n, w, g, fp8, M):
    """Steps that move more than 512 MB (runs of items per XCD), two of them;
    windows at both ends and in between."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    wt = (0.02 * torch.randn(n, generator=gen, device="cuda")).to(DT["f32" if w == "f32" else "bf16"])
    grad = (1e-2 * torch.randn(M, n, generator=gen, device="cuda")).to(DT[g])
    p = sm.ParamBuffers.with_state(wt, grad, fp8=fp8, master=w == "master", weight_decay=0.1)
    small = Case(700, "f32", "f32", False, M=M)
    cfg = sm.AdamWConfig(lr=1e-3, beta2=0.99, seed=n, rounding=sm.ROUND_STOCHASTIC)
    pset = sm.ParamSet([small.buffers(), p], M=M)
    ends = [(0, 5000), (n // 2 // 256 * 256, 7000), ((n - 4000) // 256 * 256, None)]
    views = [Window(p, M, a, k or n - a) for a, k in ends]
    for t in (1, 2):
        e = [v.expect(cfg, t, 1) for v in views]
        es = small.expect(cfg, t, 0)
        sm.adamw(cfg, pset, t)
        torch.cuda.synchronize()
        for v, x in zip(views, e):
            v.check(x, (t, v.base))
        small.check(es, t)


@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_nan_and_infinite_gradients_stay_where_they_are(gpu_lib, fp8):
    """Without a clipping factor a NaN gradient spoils its own entry only, and
    an infinite one too; the others of its block are as without it."""
    a, b = (Case(600, "f32", "f32", fp8, zero=True) for _ in range(2))
    bad = [3, 299, 599]
    for c in (a, b):
        c.grad[0, bad] = 0.0
    a.grad[0, 3], a.grad[0, 299], a.grad[0, 599] = float("nan"), float("inf"), float("-inf")
    keep = np.setdiff1d(np.arange(600), bad)
    cfg = sm.AdamWConfig(lr=1e-3, seed=5)
    for c in (a, b):
        ps = sm.ParamSet([c.buffers()])
        for t in (1, 2):
            sm.adamw(cfg, ps, t)
    torch.cuda.synchronize()
    assert not np.isfinite(np64(a.w)[bad]).any()
    for x, y in zip(a.written(), b.written()):
        x, y = np64(x.float()), np64(y.float())
        if len(x) == 600:
            x, y = x[keep], y[keep]
        assert np.array_equal(x, y)
    assert np.isnan(np64(a.m.float())[bad]).all() or not fp8
    assert not np.isfinite(np64(a.v.float())[bad]).any()


def test_extreme_magnitudes(gpu_lib):
    """Zero, denormal and very large gradients and moments in one block, and
    blocks of nothing else."""
    for fp8 in (False, True):
        cs = []
        for size in (0.0, 1e-30, 1e-19, 1.0, 1e15):
            c = Case(520, "f32", "f32", fp8, zero=True, gsize=size)
            c.grad[0, 17] = 1e-22
            c.grad[0, 18] = 0.0
            cs.append(c)
        run_and_check(cs, t=1, steps=2, eps=1e-10)


def test_small_second_moments_keep_the_smallest_code(gpu_lib):
    """Gradients from 1 to 1e-9 in one block: second moments far below the
    codes' range take the smallest code, zero ones stay zero, and the weights
    move by at most a few lr (m / sqrt(v) would be huge with v lost)."""
    c = Case(1024, "f32", "f32", True, zero=True)
    c.grad[0] = torch.tensor([10.0 ** -(i % 10) for i in range(1024)]).cuda()
    c.grad[0, 512:768:7] = 0.0
    pset = run_and_check([c], t=1, steps=4)
    code = c.v.view(torch.uint8).cpu().numpy()
    g = c.grad[0].cpu().numpy()
    assert np.all(code[g > 0] >= 1) and np.any(code[g > 0] == 1) and np.all(code[g == 0] == 0)
    before = np64(c.w)
    for t in range(5, 25):
        sm.adamw(sm.AdamWConfig(lr=1e-3, beta2=0.99, seed=t), pset, t)
    assert np.all(np.abs(np64(c.w) - before) <= 20 * 1e-3 * 4)


# ---------------------------------------------------------------- skipping, device-side index

def _snapshot(cases):
    return [[raw(t).copy() for t in c.written()] for c in cases]


@pytest.mark.parametrize("which", ["gscale", "lr_scale"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_factor_that_is_not_finite_skips_the_step(gpu_lib, which, value):
    cases = [Case(n, "master", "bf16", f) for n in (100, 3000) for f in (False, True)]
    pset = sm.ParamSet([c.buffers() for c in cases])
    before = _snapshot(cases)
    bad = torch.tensor(value, device="cuda")
    step = torch.tensor([41], dtype=torch.int64, device="cuda")
    sm.adamw(sm.AdamWConfig(), pset, 3, **{which: bad})
    sm.adamw(sm.AdamWConfig(), pset, step=step, **{which: bad})
    torch.cuda.synchronize()
    assert int(step) == 41
    for x, y in zip(before, _snapshot(cases)):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))
    step.fill_(-7)                     # not a number of steps: skipped as well
    sm.adamw(sm.AdamWConfig(), pset, step=step)
    torch.cuda.synchronize()
    assert int(step) == -7
    for x, y in zip(before, _snapshot(cases)):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))
    step.fill_(41)
    sm.adamw(sm.AdamWConfig(), pset, step=step)
    torch.cuda.synchronize()
    assert int(step) == 42


@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_device_index_and_schedule_equal_the_host_ones(gpu_lib, fp8):
    a, b = ([Case(n, "bf16", "bf16", fp8) for n in (90, 5000)] for _ in range(2))
    cfg = sm.AdamWConfig(lr=4e-3, rounding=sm.ROUND_STOCHASTIC, seed=3)
    pa, pb = (sm.ParamSet([c.buffers() for c in x]) for x in (a, b))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    ls = torch.ones(1, device="cuda")
    for t in range(1, 6):
        ls.fill_(2.0 ** -t)     # exact: lr * ls is the float that the host passes
        sm.adamw(cfg, pa, step=step, lr_scale=ls)
        half = sm.AdamWConfig(lr=4e-3 * 2.0 ** -t, rounding=sm.ROUND_STOCHASTIC, seed=3)
        sm.adamw(half, pb, t)
    torch.cuda.synchronize()
    for x, y in zip(_snapshot(a), _snapshot(b)):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))


def test_calls_repeat_bit_for_bit(gpu_lib):
    snaps = []
    for _ in range(2):
        cases = [Case(n, "bf16", "bf16", f, M=3) for n in (700, 9000) for f in (False, True)]
        ps = sm.ParamSet([c.buffers() for c in cases], M=3)
        for t in range(1, 4):
            out = sm.grad_norm([ps], 0.5)
            sm.adamw(sm.AdamWConfig(rounding=sm.ROUND_STOCHASTIC, seed=8), ps, t, gscale=out[1:])
        torch.cuda.synchronize()
        snaps.append((_snapshot(cases), out.cpu()))
    assert torch.equal(snaps[0][1], snaps[1][1])
    for x, y in zip(snaps[0][0], snaps[1][0]):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_captured_steps_replay_as_a_training_loop(gpu_lib, fp8):
    """Norm and step captured once (their index and schedule on the device),
    replayed with eager work and synchronizations between, every replay equal
    to the eager loop's step; one replay's gradient is not finite."""
    def make():
        cs = [Case(n, "bf16", "bf16", fp8) for n in (33, 2048, 7000)]
        return cs, sm.ParamSet([c.buffers() for c in cs])
    eager, pe = make()
    graphed, pg = make()
    cfg = sm.AdamWConfig(lr=3e-3, rounding=sm.ROUND_STOCHASTIC, seed=17)
    se, sg = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    oe, og = (torch.zeros(2, device="cuda") for _ in range(2))
    ls = torch.ones(1, device="cuda")

    def one(ps, out, step):
        sm.grad_norm([ps], 1.0, out=out)
        sm.adamw(cfg, ps, step=step, gscale=out[1:], lr_scale=ls)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one(pg, og, sg)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    side = torch.randn(256, 256, device="cuda")
    for k in range(6):
        for a, b in zip(eager, graphed):
            x = 0.03 * torch.randn(a.grad.shape, generator=gen, device="cuda")
            if k == 3:
                x[0, 5] = float("inf")
            a.grad.copy_(x)
            b.grad.copy_(x)
        ls.fill_(1.0 / (k + 1))
        graph.replay()
        one(pe, oe, se)
        side = torch.tanh(side @ side.T * 1e-3)
        torch.cuda.synchronize()
        assert int(se) == int(sg) == (k + 1 if k < 3 else k)
        assert np.array_equal(raw(oe), raw(og))
        for x, y in zip(_snapshot(eager), _snapshot(graphed)):
            assert all(np.array_equal(p, q) for p, q in zip(x, y)), k


def test_sets_are_refused_inside_a_capture(gpu_lib):
    c = Case(64)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    sm.ParamSet([c.buffers()], ws=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(sm.SmError) as e:
            sm.ParamSet([c.buffers()], ws=ws)
        assert e.value.code == 5


def test_other_streams(gpu_lib):
    """A set made on one stream, used on others in order."""
    a, b = Case(50000, "bf16", "bf16", True), Case(50000, "bf16", "bf16", True)
    pa, pb = sm.ParamSet([a.buffers()]), sm.ParamSet([b.buffers()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    cfg = sm.AdamWConfig(seed=2)
    for t in range(1, 7):
        s = streams[t % 2]
        s.wait_stream(streams[1 - t % 2])
        with torch.cuda.stream(s):
            out = sm.grad_norm([pa], 1.0)
            sm.adamw(cfg, pa, t, gscale=out[1:])
        out = sm.grad_norm([pb], 1.0)
        sm.adamw(cfg, pb, t, gscale=out[1:])
    torch.cuda.synchronize()
    for x, y in zip(a.written(), b.written()):
        assert np.array_equal(raw(x), raw(y))


def test_shapes_rows_and_shared_gradients(gpu_lib):
    """Weights of any rank, gradients with and without the leading 1, two
    parameters on one gradient, a workspace of the caller's: all as flat ones."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    g = 0.01 * torch.randn(6, 5, 41, generator=gen, device="cuda")

    def params(shapes):
        out = []
        for k, (ws, gs) in enumerate(shapes):
            p = sm.ParamBuffers.with_state(torch.full(ws, 0.5, device="cuda"), g.view(gs),
                                           fp8=k % 2 == 1)
            out.append(p)
        return out

    n = g.numel()
    cfg = sm.AdamWConfig(seed=4)
    results = []
    for shapes in ([((6, 5, 41), (6, 5, 41)), ((6, 205), (1, 6, 205)), ((n,), (1, n))],
                   [((n,), (n,))] * 3):
        ps = params(shapes)
        ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
        pset = sm.ParamSet(ps, ws=ws)
        for t in (1, 2):
            sm.adamw(cfg, pset, t)
        norm = sm.grad_norm([pset], 1.0)
        torch.cuda.synchronize()
        results.append([raw(x) for p in ps for x in (p.w, p.m, p.v)] + [raw(norm)])
    assert all(np.array_equal(a, b) for a, b in zip(*results))
    assert abs(float(norm[0]) - float((3 * g.double().square().sum()).sqrt())) < 1e-5


def test_hyper_parameters_at_their_ends(gpu_lib):
    """No averaging, no decay, no schedule, eps from 1e-15 to large, far steps."""
    for kw in (dict(beta1=0.0), dict(beta2=0.0), dict(beta1=0.0, beta2=0.0), dict(eps=1e-15),
               dict(eps=10.0), dict(beta1=0.999, beta2=0.99999), dict(lr=0.0)):
        run_and_check([Case(n, w, "bf16", f, wd=0.01) for n in (70, 1500) for w in ("f32", "bf16")
                       for f in (False, True)], **kw)
    run_and_check([Case(900, "f32", "f32", f) for f in (False, True)], t=(1 << 40) + 3,
                  seed=(1 << 64) - 1)


def test_schedule_factor_with_a_host_index(gpu_lib):
    a, b = ([Case(n, "f32", "f32", f, wd=0.3) for n in (90, 3000) for f in (False, True)]
            for _ in range(2))
    sm.adamw(sm.AdamWConfig(lr=1e-2), sm.ParamSet([c.buffers() for c in a]), 4,
             lr_scale=torch.tensor(0.25, device="cuda"))
    sm.adamw(sm.AdamWConfig(lr=2.5e-3), sm.ParamSet([c.buffers() for c in b]), 4)
    torch.cuda.synchronize()
    # 0.25 * float32(1e-2) is float32(2.5e-3)
    for x, y in zip(_snapshot(a), _snapshot(b)):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))


def test_two_graphs_of_one_set(gpu_lib):
    """The norm and the step captured apart, replayed in turn, with another set's
    norm joined; equal to the eager calls."""
    def make():
        a, b = Case(5000, "bf16", "bf16", True), Case(40000, "f32", "f32")
        return [a, b], sm.ParamSet([a.buffers()]), sm.ParamSet([b.grad_only()])
    cs, p1, p2 = make()
    ce, q1, q2 = make()
    out = torch.zeros(2, device="cuda")
    step, step_e = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    cfg = sm.AdamWConfig(seed=21, rounding=sm.ROUND_STOCHASTIC)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        sm.grad_norm([p1, p2], 0.3, scale=0.5, out=out)
    with torch.cuda.graph(g2):
        sm.adamw(cfg, p1, step=step, gscale=out[1:])
    for k in range(5):
        for a, b in zip(cs, ce):
            x = torch.randn_like(a.grad.float()) * 0.01
            a.grad.copy_(x)
            b.grad.copy_(x)
        g1.replay()
        g2.replay()
        o = sm.grad_norm([q1, q2], 0.3, scale=0.5)
        sm.adamw(cfg, q1, step=step_e, gscale=o[1:])
        torch.cuda.synchronize()
        assert torch.equal(o, out) and int(step) == k + 1
        assert all(np.array_equal(p, q) for p, q in zip(_snapshot(cs)[0], _snapshot(ce)[0]))


def test_a_set_made_and_dropped_on_side_streams(gpu_lib):
    """Sets whose tables belong to one stream, used on another and dropped at
    once, while the first stream allocates over what it gets back."""
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = Case(200000, "bf16", "bf16", True), Case(200000, "bf16", "bf16", True)
    torch.cuda.synchronize()
    cfg = sm.AdamWConfig(seed=1)
    pb = sm.ParamSet([b.buffers()])
    for t in range(1, 9):
        with torch.cuda.stream(s1):
            ps = sm.ParamSet([a.buffers()])
        with torch.cuda.stream(s2):
            sm.adamw(cfg, ps, t)
        del ps
        with torch.cuda.stream(s1):
            for _ in range(4):
                torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
        sm.adamw(cfg, pb, t)
    torch.cuda.synchronize()
    for x, y in zip(a.written(), b.written()):
        assert np.array_equal(raw(x), raw(y))


def test_refusals_of_a_live_set(gpu_lib):
    c = Case(64)
    ps = sm.ParamSet([c.buffers()])
    only = sm.ParamSet([c.grad_only()])
    ok = sm.AdamWConfig()
    before = _snapshot([c])
    one = torch.ones(1, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def code(fn):
        with pytest.raises(sm.SmError) as e:
            fn()
        return e.value.code

    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-16),
                dict(eps=float("inf")), dict(rounding=2)):
        assert code(lambda: sm.adamw(sm.AdamWConfig(**bad), ps, 1)) == 1, bad
    assert code(lambda: sm.adamw(ok, only, 1)) == 1          # gradients alone
    for kw in (dict(), dict(t=1, step=step), dict(t=0), dict(t=-1)):
        with pytest.raises(ValueError):
            sm.adamw(ok, ps, **kw)
    for kw in (dict(gscale=torch.ones(2, device="cuda")), dict(gscale=one.double()),
               dict(gscale=torch.ones(1)), dict(lr_scale=one.half())):
        with pytest.raises(ValueError):
            sm.adamw(ok, ps, 1, **kw)
    with pytest.raises(ValueError, match="step must be"):
        sm.adamw(ok, ps, step=step.int())
    for kw in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("nan")),
               dict(max_norm=1.0, scale=float("inf"))):
        assert code(lambda: sm.grad_norm([ps], **kw)) == 1, kw
    assert code(lambda: sm.grad_norm([ps] * 9, 1.0)) == 5
    assert code(lambda: sm.grad_norm([ps, only, ps], 1.0)) == 1
    with pytest.raises(ValueError, match="out must have shape"):
        sm.grad_norm([ps], 1.0, out=torch.zeros(3, device="cuda"))
    ps.close()
    with pytest.raises(RuntimeError):
        sm.adamw(ok, ps, 1)
    torch.cuda.synchronize()
    assert all(np.array_equal(p, q) for p, q in zip(before[0], _snapshot([c])[0]))


# ---------------------------------------------------------------- gradient norm

def _norm_ok(out, sets, scale, max_norm):
    """Eight squares summed in float32 (8 roundings, and one each for the mean
    and the result): relative 10 * 2^-24, doubled for the factor."""
    norm, coef = A.grad_norm(sets, scale, max_norm)
    got = out.double().cpu().numpy()
    assert abs(got[0] - norm) <= 10 * 2.0 ** -24 * norm, (got[0], norm)
    assert abs(got[1] - coef) <= 20 * 2.0 ** -24 * abs(coef), (got[1], coef)


@pytest.mark.parametrize("max_norm", [1e-3, 0.5, 1e6, float("inf")])
def test_norm_over_sets_of_different_types(gpu_lib, max_norm):
    groups = [(1, [Case(n, "f32", "f32") for n in LENGTHS]),
              (3, [Case(n, "bf16", "bf16", M=3, stride=n + s) for n in (5, 2000, 9001)
                   for s in (0, 3)]),
              (2, [Case(n, "f32", "f32", M=2, shift=1) for n in (257, 4000)])]
    sets = [sm.ParamSet([c.grad_only() if i % 2 else c.buffers() for i, c in enumerate(cs)], M=M)
            for M, cs in groups]
    want = [(M, [c.grads64() for c in cs]) for M, cs in groups]
    for scale in (1.0, 2.0 ** -10, -3.0, 0.0):
        _norm_ok(sm.grad_norm(sets, max_norm, scale=scale), want, scale, max_norm)
    _norm_ok(sm.grad_norm(sets[1:2], max_norm), want[1:2], 1.0, max_norm)


def test_norm_of_many_entries(gpu_lib):
    """2^26 + 13 entries of one magnitude: a float32 sum would stop growing."""
    n = (1 << 26) + 13
    g = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    out = sm.grad_norm([sm.ParamSet([sm.ParamBuffers(grad=g)])], 1.0)
    norm = 0.5 * np.sqrt(float(n))
    assert abs(float(out[0]) - norm) <= 10 * 2.0 ** -24 * norm


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 1e25])
def test_norm_that_is_not_finite_gives_no_factor(gpu_lib, bad):
    c = Case(5000)
    c.grad[0, 4321] = bad
    out = sm.grad_norm([sm.ParamSet([c.grad_only()])], 1.0)
    assert not np.isfinite(float(out[0])) and np.isnan(float(out[1]))


def test_norm_of_nothing(gpu_lib):
    sets = [sm.ParamSet([sm.ParamBuffers(grad=torch.zeros(n, device="cuda"))]) for n in (0, 5, 0)]
    for s in ([sets[0]], [sets[1]], sets):
        out = sm.grad_norm(s, 2.0, scale=0.5)
        assert out.tolist() == [0.0, 0.5]
    three = sm.ParamSet([sm.ParamBuffers(grad=torch.full((9,), 1.0, device="cuda"))])
    assert sm.grad_norm([sets[0], three, sets[2]], float("inf")).tolist() == [3.0, 1.0]


# One worker's norm takes at most 512 workgroups, each several items here.
def test_norms_repeat_over_many_workgroups(gpu_lib):
    """2048 workgroups and more items than that: every call gives the same
    bits, whichever workgroup joins the sums, and leaves the counter ready."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    g = torch.randn(50_000_003, generator=gen, device="cuda")
    ps = sm.ParamSet([sm.ParamBuffers(grad=g)])
    outs = torch.stack([sm.grad_norm([ps], 1.0) for _ in range(50)])
    want = float(g.double().square().sum().sqrt())
    assert torch.equal(outs, outs[:1].expand(50, 2))
    assert abs(float(outs[0, 0]) - want) <= 10 * 2.0 ** -24 * want


# ---------------------------------------------------------------- 8-bit states

@pytest.mark.parametrize("n", [1, 7, 256, 257, 2048, 2305, 100003, 0])
def test_pack_and_unpack(gpu_lib, n):
    """Codes and scales equal the oracle's, the values come back exactly, and
    packing those again gives the same values."""
    rng = np.random.default_rng(n)
    size = np.exp(4 * rng.standard_normal(n)) * 1e-4
    m = (size * rng.standard_normal(n)).astype(np.float32)
    v = (size ** 2 * rng.standard_normal(n) ** 2).astype(np.float32)
    if n > 4:
        m[:3] = [0.0, -0.0, 1e-42]
        v[:3] = [0.0, 1e-42, 3e-39]
    for shift in (0, 1):     # aligned and element-aligned inputs
        dm, dv = (torch.cat([torch.zeros(shift), torch.from_numpy(x)]).cuda()[shift:]
                  for x in (m, v))
        m8, v8, ms, vs = sm.state8_pack(dm, dv)
        torch.cuda.synchronize()
        for x, kind, code, scale in ((m, "m", m8, ms), (v, "v", v8, vs)):
            want, s = A.pack(x.astype(np.float64), kind) if n else (np.zeros(0), np.zeros(0))
            assert np.array_equal(np64(scale), s), kind
            assert np.array_equal(np64(code.float()), want), kind
        um, uv = sm.state8_unpack(m8, v8, ms, vs)
        assert np.array_equal(np64(um), np64(m8.float()) * A.per_entry(np64(ms), n))
        assert np.array_equal(np64(uv), np64(v8.float()) * A.per_entry(np64(vs), n))
        again = sm.state8_unpack(*sm.state8_pack(um, uv))
        assert torch.equal(again[0], um) and torch.equal(again[1], uv)


def test_pack_of_values_that_are_not_finite(gpu_lib):
    m = torch.linspace(-1, 1, 300)
    v = torch.linspace(0, 2, 300)
    clean = sm.state8_pack(m.cuda(), v.cuda())
    m2, v2 = m.clone(), v.clone()
    m2[[3, 4, 290]] = torch.tensor([float("nan"), float("inf"), float("-inf")])
    v2[[5, 6, 7, 291]] = torch.tensor([float("nan"), float("inf"), -1.0, float("-inf")])
    got = sm.state8_pack(m2.cuda(), v2.cuda())
    gm, gv = sm.state8_unpack(*got)
    assert torch.isnan(gm[[3, 4, 290]]).all()
    assert torch.isnan(gv[5]) and torch.isposinf(gv[6]) and gv[7] == 0 and gv[291] == 0
    km, kv = (np.setdiff1d(np.arange(300), i) for i in ([3, 4, 290], [5, 6, 7, 291]))
    assert np.array_equal(np64(got[0].float())[km], np64(clean[0].float())[km])
    assert np.array_equal(np64(got[1].float())[kv], np64(clean[1].float())[kv])
    assert torch.equal(got[2], clean[2]) and torch.equal(got[3], clean[3])


def test_states_taken_into_8_bits_go_on(gpu_lib):
    """A run that changes from float32 to 8-bit states: one more step of both
    from the same moments moves the weights alike, to the states' rounding.
    m carries a relative 2^-4 of itself, so an entry's change of 0.1 m-parts
    and new gradient differs by at most 2^-4 |b1 m| + 2^-10 of the block's
    largest (subnormal codes), through sqrt(v) to 2^-3 / 2 on top."""
    n = 3000
    rng = np.random.default_rng(12)
    c = Case(n, "f32", "f32", False, gen=rng)
    m8, v8, ms, vs = sm.state8_pack(c.m.clone(), c.v.clone())
    w8 = c.w.clone()
    q = sm.ParamBuffers(grad=c.grad, w=w8, m=m8, v=v8, m_scale=ms, v_scale=vs)
    w0, m0 = np64(c.w), np64(c.m)
    sc = A.per_entry(np64(ms), n)
    cfg = sm.AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.99)
    sm.adamw(cfg, sm.ParamSet([c.buffers()]), 50)
    sm.adamw(cfg, sm.ParamSet([q]), 50)
    torch.cuda.synchronize()
    d32, d8 = np64(c.w) - w0, np64(w8) - w0
    v1 = np64(c.v)
    den = np.sqrt(v1 / (1 - A.f32(0.99) ** 50))
    lr1 = 1e-3 / (1 - 0.9 ** 50)
    off = 0.9 * (2.0 ** -4 * np.abs(m0) + 2.0 ** -10 * sc)
    # sqrt(v8/v) lies within 1 +- 2^-3 (v of these blocks stays above the subnormal codes)
    tol = lr1 * off / den / (1 - 2.0 ** -3) + np.abs(d32) * 2.0 ** -3 + 2.0 ** -22 * np.abs(w0)
    assert np.all(np.abs(d8 - d32) <= tol)


# ---------------------------------------------------------------- together

def test_a_training_step_with_muon_and_adamw(gpu_lib):
    """A step as a run makes it: Sign-Muon on the matrices, the global norm
    over all gradients, AdamW with 8-bit states on an embedding and float32
    ones on the vectors; three steps, every AdamW tensor against the oracle,
    and the matrices as the same Muon steps alone leave them."""
    M, d = 3, 128
    rng = np.random.default_rng(77)
    bf = torch.bfloat16
    shapes = W.gpt2_block_shapes(d, 1)

    def muon():
        r = np.random.default_rng(78)
        mats = []
        for m, n in shapes:
            f = lambda *s: torch.from_numpy((0.02 * r.standard_normal(s)).astype(np.float32))
            mats.append(sm.MatrixBuffers(w=f(m, n).cuda().to(bf),
                                         mom=torch.zeros(M, m, n, device="cuda", dtype=bf),
                                         grad=f(M, m, n).cuda().to(bf)))
        return mats

    mats, alone = muon(), muon()
    cfg = sm.StepConfig(algo=sm.SIGN_MUON, M=M, wdt=bf, mdt=bf, gdt=bf, lr=1e-3)
    step, step_alone = sm.StepCall(cfg, mats), sm.StepCall(cfg, alone)
    emb = Case(1000 * d + 5, "master", "bf16", True, M=M, wd=0.1, gen=rng)
    vecs = [Case(k * d, "f32", "f32", False, M=M, gen=rng) for k in (1, 1, 3, 1, 4, 1)]
    cases = [emb] + vecs
    pset = sm.ParamSet([c.buffers() for c in cases], M=M)
    matset = sm.ParamSet([sm.ParamBuffers(grad=mb.grad) for mb in mats], M=M)
    acfg = sm.AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.95, seed=6)
    for t in range(1, 4):
        out = sm.grad_norm([matset, pset], 1.0)
        torch.cuda.synchronize()
        _norm_ok(out, [(M, [mb.grad.double().cpu().numpy().reshape(M, -1) for mb in mats]),
                       (M, [c.grads64() for c in cases])], 1.0, 1.0)
        e = [c.expect(acfg, t, i, float(out[1])) for i, c in enumerate(cases)]
        step(t)
        sm.adamw(acfg, pset, t, gscale=out[1:])
        step_alone(t)
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            c.check(e[i], (t, i))
        for a, b in zip(mats, alone):
            assert torch.equal(a.w.view(torch.int16), b.w.view(torch.int16))
            assert torch.equal(a.mom.view(torch.int16), b.mom.view(torch.int16))


def test_kernel_times_are_accounted(gpu_lib):
    c = Case(5000, "bf16", "bf16", True)
    ps = sm.ParamSet([c.buffers()])
    sm.profile_enable(True)
    try:
        sm.profile_reset()
        sm.grad_norm([ps], 1.0)
        sm.adamw(sm.AdamWConfig(), ps, 1)
        sm.state8_unpack(*sm.state8_pack(torch.ones(10, device="cuda"),
                                         torch.ones(10, device="cuda")))
        for kind, least in (("adamw", 10.0 * 5000), ("grad_norm", 2.0 * 5000), ("state8", 200.0)):
            ms, n, work = sm.profile_read(kind)
            assert n >= 1 and ms > 0 and work >= least
    finally:
        sm.profile_enable(False)


# ---------------------------------------------------------------- what graphs hold

@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_a_graph_outlives_the_references_to_its_set(gpu_lib, fp8):
    """Norm and step captured, the set's last reference dropped and memory of
    its tables' size written over and over: the replays equal the eager loop's
    steps; close() lets the set go."""
    def make():
        cs = [Case(n, "bf16", "bf16", fp8) for n in (33, 2048, 7000)]
        return cs, sm.ParamSet([c.buffers() for c in cs])
    eager, pe = make()
    graphed, pg = make()
    cfg = sm.AdamWConfig(lr=3e-3, rounding=sm.ROUND_STOCHASTIC, seed=23)
    se, sg = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    out = torch.zeros(2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sm.grad_norm([pg], 1.0, out=out)
        sm.adamw(cfg, pg, step=sg, gscale=out[1:])
    size, alive = pg.ws.numel(), weakref.ref(pg)
    del pg
    gc.collect()
    assert alive() is not None      # else a replay would run on freed tables
    for k in range(4):
        for _ in range(4):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        for a, b in zip(eager, graphed):
            x = 0.03 * torch.randn_like(a.grad.float())
            a.grad.copy_(x)
            b.grad.copy_(x)
        graph.replay()
        o = sm.grad_norm([pe], 1.0)
        sm.adamw(cfg, pe, step=se, gscale=o[1:])
        torch.cuda.synchronize()
        assert int(se) == int(sg) == k + 1 and torch.equal(o, out)
        for x, y in zip(_snapshot(eager), _snapshot(graphed)):
            assert all(np.array_equal(p, q) for p, q in zip(x, y)), k
    del graph
    alive().close()
    gc.collect()
    assert alive() is None


# ---------------------------------------------------------------- tiny and huge eps

@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_second_moments_below_the_normal_range_count_beside_a_tiny_eps(gpu_lib, fp8):
    """beta2 = 0.99999 and t = 1: v = 1e-5 g^2 from 9e-41 to 1e-37, across
    2^-126, whose root times 316 is up to a tenth of eps = 1e-15.  v is held
    to 2^-149 / 9e-41 = 2^-16 of itself at worst, half of that in the root,
    which is 0.3 % of the denominator there: 2^-26 of the change."""
    c = Case(600, "f32", "f32", fp8, zero=True)
    c.grad[0] = torch.from_numpy(np.geomspace(3e-18, 1e-16, 600).astype(np.float32)).cuda()
    run_and_check([c], t=1, lr=0.1, beta2=0.99999, eps=1e-15)


@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_the_change_under_a_huge_eps(gpu_lib, fp8):
    """eps beyond 2^126, whose reciprocal is below the normal range: the change
    is m / eps all the same (weights of 0 show it)."""
    c = Case(600, "f32", "f32", fp8, zero=True, gsize=1e18)
    c.w.zero_()
    run_and_check([c], t=1, lr=1.0, eps=2e38)


# ---------------------------------------------------------------- large sums of workers

@pytest.mark.parametrize("M", [2, 3, 64])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_step_on_a_mean_whose_sum_leaves_float32(gpu_lib, M, g):
    """Gradients of 1e38 to 3e38 of one sign: their sum is beyond float32, the
    mean, and gscale times it, are not.  The roundings are the usual ones."""
    cases = []
    for i, (n, fp8) in enumerate((n, f) for n in (7, 1030) for f in (False, True)):
        c = Case(n, "f32", g, fp8, M=M)
        x = np.random.default_rng(i).uniform(1e38, 3e38, (M, n)) * np.where(np.arange(n) % 3, 1, -1)
        c.grad.copy_(torch.from_numpy(x.astype(np.float32)))
        cases.append(c)
    run_and_check(cases, M=M, gscale=1e-38 * 2.0)


@pytest.mark.parametrize("M", [2, 3, 64])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_norm_of_a_mean_whose_sum_squared_leaves_float32(gpu_lib, M, g):
    """Entries up to 1.2e19: the mean's squares stay below 3.4e38, the sum's do
    not (M = 2: 5.8e38).  8 of them may not be added in float32 either, so
    that large entries stand alone among small ones."""
    n = 5003
    c = Case(n, "f32", g, M=M, gsize=1e12)
    c.grad[:, ::64] = 1.2e19
    out = sm.grad_norm([sm.ParamSet([c.grad_only()], M=M)], float("inf"), scale=2.0 ** -60)
    _norm_ok(out, [(M, [c.grads64()])], 2.0 ** -60, float("inf"))


# ---------------------------------------------------------------- small decays

@pytest.mark.parametrize("lr,wd", [(1e-6, 0.1), (3e-7, 0.2), (1e-4, 0.01)])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
@pytest.mark.parametrize("w", ["f32", "master"])
def test_a_small_decay_is_rounded_with_the_weight_alone(gpu_lib, lr, wd, fp8, w):
    """No gradient and no moments: a weight is w (1 - lr wd), rounded once, at
    most half a float32 step of w (and the product's own rounding, 2^-22 of
    the decay) off."""
    c = Case(2500, w, "f32", fp8, zero=True, wd=wd)
    c.grad.zero_()
    kept = c.w if c.master is None else c.master
    before = np64(kept)
    sm.adamw(sm.AdamWConfig(lr=lr), sm.ParamSet([c.buffers()]), 3)
    torch.cuda.synchronize()
    decay = A.f32(lr) * A.f32(wd)
    half = np.spacing(np.abs(before).astype(np.float32)).astype(float) / 2
    off = np.abs(np64(kept) - before * (1 - decay))
    assert np.all(off <= half + 2.0 ** -22 * decay * np.abs(before))


@pytest.mark.parametrize("wd", [0.0, 0.1])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
@pytest.mark.parametrize("w", ["f32", "bf16", "master"])
def test_an_infinite_weight_stays_one(gpu_lib, w, fp8, wd):
    c = Case(900, w, "bf16", fp8, wd=wd)
    for t in (c.w, c.master):
        if t is not None:
            t[5], t[700] = float("inf"), float("-inf")
    sm.adamw(sm.AdamWConfig(lr=1e-2), sm.ParamSet([c.buffers()]), 3)
    torch.cuda.synchronize()
    for t in (c.w, c.master):
        if t is not None:
            x = np64(t)
            assert x[5] == np.inf and x[700] == -np.inf and np.isfinite(x).sum() == 898


# ---------------------------------------------------------------- slow averages

def test_averages_too_slow_for_8_bit_states_are_refused(gpu_lib):
    """Above 0.99999 such a moment would stand still; float32 states take any
    beta below 1, and so does the limit itself."""
    c8, c32 = Case(600, "f32", "f32", True), Case(600, "f32", "f32", False)
    both = sm.ParamSet([c32.buffers(), c8.buffers()])
    before = _snapshot([c8, c32])
    for kw in (dict(beta2=0.999999), dict(beta1=0.999999), dict(beta2=0.999991)):
        with pytest.raises(sm.SmError) as e:
            sm.adamw(sm.AdamWConfig(**kw), both, 1)
        assert e.value.code == 5, kw
    torch.cuda.synchronize()
    for x, y in zip(before, _snapshot([c8, c32])):
        assert all(np.array_equal(p, q) for p, q in zip(x, y))
    del both
    run_and_check([c8], beta1=0.99999, beta2=0.99999)
    run_and_check([c32], beta1=0.999999, beta2=0.999999)


# ---------------------------------------------------------------- accounting

def test_small_launches_are_accounted_as_well(gpu_lib):
    """The tables' fill and the kernel of a device-side step index: kind misc."""
    cases = [Case(40 + i) for i in range(70)]      # three fills
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    sm.profile_enable(True)
    try:
        sm.profile_reset()
        ps = sm.ParamSet([c.buffers() for c in cases])
        assert sm.profile_read("misc")[1] == 3
        sm.adamw(sm.AdamWConfig(), ps, step=step)
        ms, n, work = sm.profile_read("misc")
        assert n == 4 and ms > 0 and work >= 70 * (88 + 16) + 16
        assert sm.profile_read("adamw")[1] == 1
    finally:
        sm.profile_enable(False)


def test_captured_launches_are_not_accounted(gpu_lib):
    """Norm and step captured while the accounting is on: the totals are the
    eager calls', and the graph replays."""
    c = Case(5000, "bf16", "bf16", True)
    ps = sm.ParamSet([c.buffers()])
    out = torch.zeros(2, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def one():
        sm.grad_norm([ps], 1.0, out=out)
        sm.adamw(sm.AdamWConfig(), ps, step=step, gscale=out[1:])

    torch.cuda.synchronize()
    sm.profile_enable(True)
    try:
        sm.profile_reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one()
        for _ in range(3):
            graph.replay()
            one()
        torch.cuda.synchronize()
        assert int(step) == 6
        for kind in ("grad_norm", "adamw", "misc"):
            ms, n, work = sm.profile_read(kind)
            assert n == 3 and ms > 0, kind
    finally:
        sm.profile_enable(False)


# ---------------------------------------------------------------- any alignment, far rows, two at once

@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32state", "fp8"])
def test_step_of_long_unaligned_buffers(gpu_lib, fp8, shift):
    """Whole work items, of one unit and of several, off alignment."""
    run_and_check([Case(n, w, g, fp8, shift=shift, wd=0.05)
                   for n in (6145, 20000) for w, g in (("f32", "f32"), ("master", "bf16"),
                                                       ("bf16", "bf16"), ("bf16", "f32"))])


@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_norm_of_long_unaligned_gradients(gpu_lib, g, shift):
    """One worker's whole rounds (16384 entries) and the rest at any offset."""
    cases = [Case(n, "f32", g, shift=shift) for n in (16384, 16385, 50007)]
    out = sm.grad_norm([sm.ParamSet([c.grad_only() for c in cases])], 1.0)
    _norm_ok(out, [(1, [c.grads64() for c in cases])], 1.0, 1.0)


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("n", [1, 255, 2305, 9001])
def test_conversion_of_codes_at_any_byte(gpu_lib, n, offset):
    """Codes written to and read from odd addresses: as the aligned ones, and
    nothing beside them written."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    m = torch.randn(n, generator=gen, device="cuda")
    v = torch.randn(n, generator=gen, device="cuda").square()
    m8, v8, ms, vs = sm.state8_pack(m, v)
    bufs = [torch.full((n + 16,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty_like(ms) for _ in range(2)]
    code = sm.lib().sm_state8_pack(m.data_ptr(), v.data_ptr(), n, bufs[0].data_ptr() + offset,
                                   bufs[1].data_ptr() + offset, scales[0].data_ptr(),
                                   scales[1].data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    for buf, want, scale, want_scale in zip(bufs, (m8, v8), scales, (ms, vs)):
        assert torch.equal(buf[offset:offset + n], want.view(torch.uint8))
        assert bool((buf[:offset] == 0xA5).all()) and bool((buf[offset + n:] == 0xA5).all())
        assert torch.equal(scale, want_scale)
    odd = sm.state8_unpack(bufs[0][offset:offset + n].view(m8.dtype),
                           bufs[1][offset:offset + n].view(v8.dtype), *scales)
    assert all(torch.equal(a, b) for a, b in zip(odd, sm.state8_unpack(m8, v8, ms, vs)))


def test_rows_further_apart_than_32_bits(gpu_lib):
    """Two workers' rows 2^32 + 5 entries apart: step and norm."""
    n, stride = 9000, (1 << 32) + 5
    for fp8 in (False, True):
        far, near = (Case(n, "f32", "bf16", fp8, M=2) for _ in range(2))
        buf = torch.empty(stride + n, dtype=torch.bfloat16, device="cuda")
        far.grad = torch.as_strided(buf, (2, n), (stride, 1))
        far.grad.copy_(near.grad)
        outs = []
        for c in (far, near):
            ps = sm.ParamSet([c.buffers()], M=2)
            outs.append(sm.grad_norm([ps], 1.0))
            sm.adamw(sm.AdamWConfig(seed=3), ps, 2, gscale=outs[-1][1:])
        torch.cuda.synchronize()
        assert torch.equal(*outs)
        _norm_ok(outs[0], [(2, [near.grads64()])], 1.0, 1.0)
        for x, y in zip(far.written(), near.written()):
            assert np.array_equal(raw(x), raw(y))
        del buf, far


def test_two_sets_at_once(gpu_lib):
    """Sets of their own may run on two streams at the same time."""
    def make(k):
        cs = [Case(n, "bf16", "bf16", f, wd=0.1) for n in (1000 + k, 400000 + k)
              for f in (False, True)]
        return cs, sm.ParamSet([c.buffers() for c in cs])
    at_once, alone = [make(k) for k in range(2)], [make(k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    step = torch.zeros(4, dtype=torch.int64, device="cuda")
    cfg = sm.AdamWConfig(seed=6, rounding=sm.ROUND_STOCHASTIC)
    torch.cuda.synchronize()
    outs = []
    for t in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                outs.append(sm.grad_norm([at_once[k][1]], 1.0))
                sm.adamw(cfg, at_once[k][1], step=step[k:k + 1], gscale=outs[-1][1:])
    torch.cuda.synchronize()
    for t in range(5):
        for k in range(2):
            out = sm.grad_norm([alone[k][1]], 1.0)
            sm.adamw(cfg, alone[k][1], step=step[2 + k:3 + k], gscale=out[1:])
            assert torch.equal(out, outs[2 * t + k])
    torch.cuda.synchronize()
    for (a, _), (b, _) in zip(at_once, alone):
        for x, y in zip(_snapshot(a), _snapshot(b)):
            assert all(np.array_equal(p, q) for p, q in zip(x, y))
