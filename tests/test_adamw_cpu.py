"""The AdamW operators without a GPU: the oracle against independent
implementations (torch.optim.AdamW in float64, torch's float8 conversions),
the struct layouts, and every refusal of the C ABI and the Python front end
(all on the host, before any HIP call)."""
import ctypes
import gc
import os
import subprocess
import weakref

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm
from matrix_aware_optimizer_momentum_amd import _binding as B
from oracle import adamw_oracle as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5


# ---------------------------------------------------------------- oracle pins

def test_oracle_step_is_torch_adamw():
    """float64 torch.optim.AdamW over ten steps; both use float64 arithmetic on
    hyper-parameters that are float32 values, so a relative 1e-12 holds."""
    rng = np.random.default_rng(1)
    c = dict(lr=A.f32(1e-3), beta1=A.f32(0.9), beta2=A.f32(0.99), eps=A.f32(1e-8))
    wd = A.f32(0.1)
    w = rng.standard_normal(500)
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([p], lr=c["lr"], betas=(c["beta1"], c["beta2"]), eps=c["eps"],
                            weight_decay=wd)
    m, v = np.zeros(500), np.zeros(500)
    for t in range(1, 11):
        g = rng.standard_normal(500)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        _, m, v = A.moments(g[None], m, v, c)
        w, _ = A.weights(w, m, v, t, c, wd=wd)
    assert np.max(np.abs(w - p.detach().numpy())) <= 1e-12 * np.max(np.abs(w))


@pytest.mark.parametrize("kind,dt", [("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)])
def test_oracle_grid_is_torch_float8(kind, dt):
    """Every code, and values between codes, against torch's conversions."""
    codes = torch.arange(0, 127 if kind == "m" else 124, dtype=torch.uint8).view(dt).float().numpy()
    codes = codes.astype(np.float64)
    assert codes.max() == A.KINDS[kind][3]
    assert np.array_equal(A.to_grid(codes, kind), codes)
    x = np.concatenate([codes[:-1] + f * np.diff(codes) for f in (0.25, 0.4999, 0.5, 0.5001)])
    want = torch.from_numpy(x.astype(np.float32)).to(dt).float().numpy()
    assert np.array_equal(A.to_grid(x.astype(np.float32).astype(np.float64), kind), want)


def test_stochastic_grid_is_unbiased_and_random_bits_are_uniform():
    """Bits: every one of the 32 set in half of 2^18 entries (5 sigma of a fair
    coin), low and high halves uncorrelated; the grid's mean over them is the
    value (5 sigma of the rounding's deviation, at most half a step)."""
    n = 1 << 18
    r, rw = A.random_bits(7, 3, 2, np.arange(n))
    for k in range(32):
        assert abs(((r >> np.uint64(k)) & np.uint64(1)).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
    lo, hi = (r & np.uint64(0xFFFF)).astype(float), (r >> np.uint64(16)).astype(float)
    for a, b in ((lo, hi), (lo, rw.astype(float)), (hi, rw.astype(float)), (lo[1:], lo[:-1])):
        assert abs(np.corrcoef(a, b)[0, 1]) < 5 / np.sqrt(n)
    for kind in ("m", "v"):
        for x in (3.3, 0.0061, 2.0 ** -9 * 0.37 if kind == "m" else 2.0 ** -16 * 0.37, 300.1):
            got = A.to_grid(np.full(n, x), kind, (lo + 0.5) / 65536)
            assert abs(got.mean() - x) < 5 * 0.5 * A.step_of(np.array([x]), kind)[0] / np.sqrt(n)
    r2, _ = A.random_bits(7, 4, 2, np.arange(n))
    r3, _ = A.random_bits(7, 3, 2, np.arange(n) + (1 << 32))
    for other in (r2, r3):
        assert (other == r).mean() < 1e-4


@pytest.mark.parametrize("kind,steps", [("v", range(5, 9)), ("m", range(9, 17))])
@pytest.mark.parametrize("beta,off", [(0.999, 0.002), (0.9999, 0.02), (0.99999, 0.2)])
def test_decaying_moments_leave_their_codes_at_the_stated_rate(kind, steps, beta, off):
    """A moment that is k of the steps below it (a power of two: of the finer
    ones) falls with a chance of (1 - beta) k, in steps of 2^-16: over all
    16-bit numbers, to 2^-17 / ((1 - beta) k), at k = 5 0.16, 1.6 and 16 %."""
    u = (np.arange(65536) + 0.5) / 65536
    for k in steps:
        x = float(k) * 2.0 ** 3
        want = (1 - beta) * k
        got = (A.to_grid(np.full(65536, beta * x), kind, u) < x).mean()
        assert abs(got - want) <= 2.0 ** -17 * 1.001 and abs(got / want - 1) < off


@pytest.mark.parametrize("kind", ["m", "v"])
def test_oracle_scale_brackets_the_largest(kind):
    largest = A.KINDS[kind][3]
    for a in (1e-30, 0.3, 1.75, 1.7500001, 2.0, 448.0, 449.0, 3e38, 1e-45):
        s = A.scale_of(float(np.float32(a)), kind)
        assert float(np.float32(a)) <= largest * s
        assert s == 2.0 ** -126 or float(np.float32(a)) > largest * s / 2
    assert A.scale_of(0.0, kind) == 2.0 ** -126


# ---------------------------------------------------------------- the boundary

def test_struct_layouts_match_c(tmp_path):
    src = tmp_path / "layout.c"
    fields = ["sizeof(sm_param)", "sizeof(sm_adamw_config)"]
    fields += [f"offsetof(sm_param, {f})" for f, _ in B.Param._fields_]
    fields += [f"offsetof(sm_adamw_config, {f})" for f, _ in B.AdamWConfig._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sm.h"\nint main(void){'
                   + "".join(f'printf("%zu ", {f});' for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", f"-I{ROOT}/include", "-I/opt/rocm/include",
                    str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [ctypes.sizeof(B.Param), ctypes.sizeof(B.AdamWConfig)]
    want += [getattr(B.Param, f).offset for f, _ in B.Param._fields_]
    want += [getattr(B.AdamWConfig, f).offset for f, _ in B.AdamWConfig._fields_]
    assert got == want


def test_kernel_kinds_match_the_library():
    lib = B.lib()
    for i, name in enumerate(B.KERNEL_KINDS):
        assert lib.sm_kernel_kind_name(i).decode() == name
    assert lib.sm_kernel_kind_name(len(B.KERNEL_KINDS)) == b"unknown"


def _param(**kw):
    d = dict(count=100, grad_stride=100, w=0x10000, master=None, grad=0x20000, m=0x30000,
             v=0x40000, m_scale=None, v_scale=None, wdt=B.F32, gdt=B.F32, state=B.STATE_F32,
             weight_decay=0.0, lr_mult=1.0)
    d.update(kw)
    return B.Param(**d)


FP8 = dict(state=B.STATE_FP8, m_scale=0x50000, v_scale=0x60000)


def _create(params, M=1, ws=0x1000000, ws_bytes=1 << 20):
    arr = (B.Param * len(params))(*params)
    h = ctypes.c_void_p(0x1234)
    code = B.lib().sm_param_set_create(arr, len(params), M, ctypes.c_void_p(ws), ws_bytes, None,
                                       ctypes.byref(h))
    assert h.value is None
    return code


@pytest.mark.parametrize("params,kw,want", [
    ([_param(count=-1)], {}, SHAPE),
    ([_param(count=(1 << 40) + 1)], {}, SHAPE),
    ([_param(count=1 << 38)], {}, SHAPE),                       # more work items than a launch
    ([_param()], dict(M=0), UNSUPPORTED),
    ([_param()], dict(M=65), UNSUPPORTED),
    ([_param()], dict(ws=0), ARG),
    ([_param()], dict(ws=0x1000010), ARG),
    ([_param()], dict(ws_bytes=64), WORKSPACE),
    ([_param(gdt=2)], {}, DTYPE),
    ([_param(wdt=2)], {}, DTYPE),
    ([_param(state=2)], {}, DTYPE),
    ([_param(grad=None)], {}, ARG),
    ([_param(grad=0x20002)], {}, ARG),
    ([_param(w=None)], {}, ARG),                                # m and v without w
    ([_param(m=None)], {}, ARG),
    ([_param(v=None)], {}, ARG),
    ([_param(w=0x10002)], {}, ARG),
    ([_param(w=0x10001, wdt=B.BF16)], {}, ARG),
    ([_param(m=0x30002)], {}, ARG),
    ([_param(m_scale=0x50000)], {}, ARG),                       # scales of float32 states
    ([_param(**{**FP8, "v_scale": None})], {}, ARG),
    ([_param(**{**FP8, "m_scale": 0x50001})], {}, ARG),
    ([_param(master=0x70000)], {}, ARG),                        # master of float32 weights
    ([_param(master=0x70002, wdt=B.BF16)], {}, ARG),
    ([_param(weight_decay=-0.1)], {}, ARG),
    ([_param(weight_decay=float("nan"))], {}, ARG),
    ([_param(lr_mult=float("inf"))], {}, ARG),
    ([_param(grad_stride=99)], dict(M=2), ARG),
    ([_param(grad_stride=(1 << 40) + 1)], dict(M=2), SHAPE),
    # overlaps: the same parameter twice, w and its gradient, moments of two
    # parameters by one entry, 8-bit scales, the workspace, a worker's row
    ([_param(), _param()], {}, ARG),
    ([_param(grad=0x10000 + 396)], {}, ARG),
    ([_param(), _param(w=0x80000, grad=0x90000, m=0x30000 + 396, v=0xA0000)], {}, ARG),
    ([_param(**{**FP8, "v_scale": 0x50000})], {}, ARG),
    ([_param(v=0x1000000)], {}, ARG),
    ([_param(w=0x20000 + 4 * 100, grad_stride=200)], dict(M=2), None),   # between the rows
    ([_param(w=0x20000 + 4 * 100, grad_stride=199)], dict(M=2), ARG),
])
def test_set_refusals(params, kw, want):
    if want is None:    # accepted by the checks: with a workspace one byte short
        arr = (B.Param * len(params))(*params)
        need = ctypes.c_size_t(0)
        assert B.lib().sm_param_set_ws(arr, len(params), ctypes.byref(need)) == 0
        assert _create(params, **{**kw, "ws_bytes": need.value - 1}) == WORKSPACE
        return
    assert _create(params, **kw) == want
    assert B.lib().sm_last_hip_error() == 0


def test_set_query_refusals():
    lib = B.lib()
    need = ctypes.c_size_t(0)
    one = (B.Param * 1)(_param())
    assert lib.sm_param_set_ws(None, 1, ctypes.byref(need)) == ARG
    assert lib.sm_param_set_ws(one, 0, ctypes.byref(need)) == ARG
    assert lib.sm_param_set_ws(one, 1, None) == ARG
    assert lib.sm_param_set_ws(one, 1, ctypes.byref(need)) == 0 and need.value % 256 == 0
    assert lib.sm_param_set_create(one, 1, 1, ctypes.c_void_p(0x1000000), 1 << 20, None,
                                   None) == ARG
    assert lib.sm_param_set_destroy(None) == 0


def test_step_and_norm_refusals_without_a_set():
    lib = B.lib()
    c = sm.AdamWConfig().c_struct()
    assert lib.sm_adamw(ctypes.byref(c), None, 1, None, None, None, None) == ARG
    assert lib.sm_adamw(None, None, 1, None, None, None, None) == ARG
    sets = (ctypes.c_void_p * 9)()
    ok = ctypes.c_void_p(0x1000000)
    assert lib.sm_grad_norm(sets, 1, 1.0, 1.0, ok, None) == ARG
    assert lib.sm_grad_norm(None, 1, 1.0, 1.0, ok, None) == ARG
    assert lib.sm_grad_norm(sets, 0, 1.0, 1.0, ok, None) == ARG
    assert lib.sm_grad_norm(sets, 1, 1.0, 1.0, None, None) == ARG
    assert lib.sm_grad_norm(sets, 1, 1.0, 1.0, ctypes.c_void_p(0x1000002), None) == ARG
    assert lib.sm_grad_norm(sets, 9, 1.0, 1.0, ok, None) == UNSUPPORTED
    assert lib.sm_last_hip_error() == 0


def test_state8_refusals():
    lib = B.lib()
    good = [0x100000, 0x200000, 1000, 0x300000, 0x400000, 0x500000, 0x600000]

    def pack(**at):
        a = list(good)
        for k, val in at.items():
            a[int(k[1:])] = val
        ptr = [a[0], a[1]] + a[3:]
        p = lib.sm_state8_pack(ptr[0], ptr[1], a[2], ptr[2], ptr[3], ptr[4], ptr[5], None)
        u = lib.sm_state8_unpack(ptr[2], ptr[3], ptr[4], ptr[5], a[2], ptr[0], ptr[1], None)
        assert p == u
        return p

    assert pack(a2=-1) == SHAPE
    assert pack(a2=(1 << 40) + 1) == SHAPE
    assert pack(a2=0, a0=None) == 0
    for i in (0, 1, 3, 4, 5, 6):
        assert pack(**{f"a{i}": None}) == ARG
    for i in (0, 1, 5, 6):
        assert pack(**{f"a{i}": good[i] + 2}) == ARG
    assert pack(a3=0x100000 + 3999) == ARG          # codes over the moments' last byte
    # two inputs may be one buffer, two outputs may not
    assert lib.sm_state8_pack(0x100000, 0x200000, 1000, 0x300000, 0x300000, 0x500000, 0x600000,
                              None) == ARG
    assert lib.sm_state8_pack(0x100000, 0x200000, 1000, 0x300000, 0x400000, 0x500000, 0x50000C,
                              None) == ARG
    assert lib.sm_last_hip_error() == 0


# ---------------------------------------------------------------- the front end

def _bufs(n=300, wdt=torch.float32, gshape=None, fp8=False, **kw):
    w = torch.zeros(n, dtype=wdt)
    return sm.ParamBuffers.with_state(w, torch.zeros(gshape or (n,), dtype=wdt), fp8=fp8, **kw)


def _edit(p, **kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("make,M,msg", [
    (lambda: _edit(_bufs(), w=torch.zeros(300, dtype=torch.float16)), 1, "must be float32 or"),
    (lambda: _edit(_bufs(), grad=torch.zeros(300, dtype=torch.float64)), 1, "must be float32 or"),
    (lambda: _bufs(gshape=(299,)), 1, "grad must have shape"),
    (lambda: _bufs(gshape=(2, 300)), 3, "grad must have shape"),
    (lambda: _bufs(), 2, "grad must have shape"),
    (lambda: _edit(_bufs(), m=None), 1, "needs m and v"),
    (lambda: _edit(_bufs(), v=torch.zeros(301)), 1, "v must have shape"),
    (lambda: _edit(_bufs(), v=torch.zeros(300, dtype=torch.bfloat16)), 1, "v must be"),
    (lambda: _edit(_bufs(), m_scale=torch.zeros(2)), 1, "have no scales"),
    (lambda: _edit(_bufs(fp8=True), m_scale=None), 1, "need m_scale"),
    (lambda: _edit(_bufs(fp8=True), v_scale=torch.zeros(1)), 1, "v_scale must have shape"),
    (lambda: _edit(_bufs(fp8=True), m=torch.zeros(300, dtype=torch.uint8)), 1, "m must be"),
    (lambda: _edit(_bufs(), master=torch.zeros(300)), 1, "only bfloat16"),
    (lambda: _edit(_bufs(wdt=torch.bfloat16), master=torch.zeros(299)), 1, "master must have"),
    (lambda: sm.ParamBuffers(grad=torch.zeros(4), m=torch.zeros(4)), 1, "m without w"),
    (lambda: sm.ParamBuffers(grad=torch.zeros(3, 4)), 2, "grad must have 2 rows"),
    (lambda: _bufs(), 1, "must be a GPU tensor"),
])
def test_front_end_refuses_before_any_pointer_crosses(make, M, msg):
    with pytest.raises(ValueError, match=msg):
        sm.ParamSet([make()], M=M)


def test_front_end_refusals_of_the_calls():
    with pytest.raises(ValueError, match="at least one parameter"):
        sm.ParamSet([])
    with pytest.raises(ValueError, match="M must be"):
        sm.ParamSet([_bufs()], M=0)
    with pytest.raises(ValueError, match="at least one set"):
        sm.grad_norm([], 1.0)
    with pytest.raises(ValueError, match="seed"):
        sm.AdamWConfig(seed=-1).c_struct()
    with pytest.raises(ValueError, match="GPU tensor"):
        sm.state8_pack(torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="v must have shape"):
        sm.state8_pack(torch.zeros(4), torch.zeros(5))
    z8 = torch.zeros(4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="m8 must be"):
        sm.state8_unpack(z8, z8, torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError, match="m_scale must have shape"):
        sm.state8_unpack(z8.view(torch.float8_e4m3fn), z8.view(torch.float8_e5m2), torch.zeros(2),
                         torch.zeros(1))


def test_with_state_makes_empty_states():
    w = torch.randn(3, 171, dtype=torch.bfloat16)
    p = sm.ParamBuffers.with_state(w, torch.zeros_like(w), fp8=True, master=True)
    assert p.m.dtype == torch.float8_e4m3fn and p.v.dtype == torch.float8_e5m2
    assert p.m.shape == p.v.shape == w.shape and p.m_scale.shape == p.v_scale.shape == (3,)
    assert not p.m.view(torch.uint8).any() and not p.v.view(torch.uint8).any()
    assert torch.equal(p.master, w.float())


# ---------------------------------------------------------------- what a set keeps alive

@pytest.fixture
def host_sets(monkeypatch):
    """ParamSet over CPU tensors: the whole front end but the GPU calls.
    capturing[0]: whether the current stream is being captured."""
    from matrix_aware_optimizer_momentum_amd import api
    capturing = [False]
    monkeypatch.setattr(api, "_check_param", lambda *a: None)
    monkeypatch.setattr(api, "_stream_of", lambda index: 0x1000)
    monkeypatch.setattr(api, "_call_on", lambda index, name, *a: None)
    monkeypatch.setattr(api, "_capturing", lambda index: capturing[0], raising=False)
    return capturing


@pytest.mark.parametrize("call", [lambda ps: sm.adamw(sm.AdamWConfig(), ps, 1),
                                  lambda ps: sm.grad_norm([ps], 1.0)], ids=["step", "norm"])
def test_a_set_of_captured_calls_is_kept_until_it_is_closed(host_sets, call):
    """A graph replays on the set's tables and buffers: they stay after the
    caller's last reference to the set, and go with close()."""
    ps = sm.ParamSet([_bufs()])
    ws, state = weakref.ref(ps.ws), weakref.ref(ps.params[0].m)
    host_sets[0] = True
    call(ps)
    host_sets[0] = False
    alive = weakref.ref(ps)
    del ps
    gc.collect()
    assert alive() is not None and ws() is not None and state() is not None
    alive().close()
    gc.collect()
    assert alive() is None and ws() is None and state() is None


def test_a_set_of_eager_calls_goes_with_its_last_reference(host_sets):
    ps = sm.ParamSet([_bufs()])
    sm.adamw(sm.AdamWConfig(), ps, 1)
    sm.grad_norm([ps], 1.0)
    alive = weakref.ref(ps)
    del ps
    gc.collect()
    assert alive() is None


def test_a_set_keeps_the_tensors_that_it_was_made_of(host_sets):
    """Its tables hold their addresses, also after a field of a ParamBuffers
    has been set anew."""
    p = _bufs(wdt=torch.bfloat16, fp8=True, master=True)
    names = ("grad", "w", "m", "v", "m_scale", "v_scale", "master")
    held = [weakref.ref(getattr(p, name)) for name in names]
    ps = sm.ParamSet([p])
    for name in names:
        setattr(p, name, getattr(p, name).clone())
    gc.collect()
    assert all(t() is not None for t in held)
    del ps
    gc.collect()
    assert all(t() is None for t in held)
