"""torch-tensor front end of libsm: same names as the C ABI, marshalling only.

Tensors must be CUDA (HIP) tensors, contiguous, float32 or bfloat16 unless
stated otherwise.  Work is enqueued on torch's current stream.  Non-OK
status codes raise SmError.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import List, Optional, Sequence

import torch

from . import _binding as B

_DT = {torch.float32: B.F32, torch.bfloat16: B.BF16}
_TORCH_DT = {B.F32: torch.float32, B.BF16: torch.bfloat16}


@dataclass
class NSParams:
    iters: int = 5
    a: float = 1.5
    b: float = -0.5
    c: float = 0.0
    eps: float = 1e-7

    def c_struct(self) -> B.NSParams:
        return B.NSParams(self.iters, self.a, self.b, self.c, self.eps)


@dataclass
class StepConfig:
    algo: int = B.SIGN_MUON
    update: int = B.UPDATE_VOTE
    M: int = 1
    wdt: torch.dtype = torch.float32
    mdt: torch.dtype = torch.float32
    gdt: torch.dtype = torch.float32
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.99
    period: int = 0
    ns: NSParams = field(default_factory=NSParams)
    gamma: float = 0.0
    cache_mode: int = B.MODE_TRIGGER
    encoding: int = B.ENC_BITS
    vote_polar: bool = False

    def c_struct(self) -> B.Config:
        return B.Config(self.algo, self.update, self.M, _DT[self.wdt], _DT[self.mdt],
                        _DT[self.gdt], self.lr, self.beta1, self.beta2, self.period,
                        self.ns.c_struct(), self.gamma, self.cache_mode, self.encoding,
                        int(self.vote_polar))


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"dtype {t.dtype} not supported (float32 / bfloat16)")
    return _DT[t.dtype]


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _expect(t: torch.Tensor, name: str, shape=None, dtype=None, min_numel=None, dev=True):
    """Shape / dtype / size check of a caller tensor before its pointer
    crosses the C ABI (which sees only raw pointers and cannot check sizes);
    then (dev) that it is a contiguous GPU tensor."""
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} must hold at least {min_numel} elements, has {t.numel()}")
    if dev:
        _dev(t, name)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ws(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _bmn(x: torch.Tensor):
    if x.dim() == 2:
        return 1, x.shape[0], x.shape[1]
    if x.dim() == 3:
        return x.shape[0], x.shape[1], x.shape[2]
    raise ValueError("expected [m, n] or [batch, m, n]")


# ------------------------------------------------------------------ sm_ns_polar

def ns_polar_ws(dtype: torch.dtype, batch: int, m: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    B.check(B.lib().sm_ns_polar_ws(_DT[dtype], batch, m, n, ctypes.byref(out)), "sm_ns_polar_ws")
    return out.value


def ns_polar(x: torch.Tensor, out: Optional[torch.Tensor] = None, normalize: bool = True,
             params: Optional[NSParams] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    _dev(x, "x")
    batch, m, n = _bmn(x)
    p = params or NSParams()
    out = torch.empty_like(x) if out is None else out
    _expect(out, "out", x.shape, x.dtype)
    ws = _ws(ns_polar_ws(x.dtype, batch, m, n), x.device, ws)
    cp = p.c_struct()
    code = B.lib().sm_ns_polar(x.data_ptr(), out.data_ptr(), _dt(x), batch, m, n,
                               int(normalize), ctypes.byref(cp), ws.data_ptr(),
                               ws.numel() * ws.element_size(), _stream())
    B.check(code, "sm_ns_polar")
    return out


def ns_polar_noalloc(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                     normalize: bool = True, params: Optional[NSParams] = None) -> torch.Tensor:
    """sm_ns_polar on the library's fixed scratch (no workspace argument).
    With out given, nothing is allocated here either."""
    _dev(x, "x")
    batch, m, n = _bmn(x)
    p = params or NSParams()
    out = torch.empty_like(x) if out is None else out
    _expect(out, "out", x.shape, x.dtype)
    cp = p.c_struct()
    code = B.lib().sm_ns_polar_noalloc(x.data_ptr(), out.data_ptr(), _dt(x), batch, m, n,
                                       int(normalize), ctypes.byref(cp), _stream())
    B.check(code, "sm_ns_polar_noalloc")
    return out


# ------------------------------------------------------------------ sm_gram_ns_cached

def gram_ns_cached_ws(dtype: torch.dtype, batch: int, m: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    B.check(B.lib().sm_gram_ns_cached_ws(_DT[dtype], batch, m, n, ctypes.byref(out)),
            "sm_gram_ns_cached_ws")
    return out.value


def gram_ns_cached(x: torch.Tensor, q: torch.Tensor, cache_state: torch.Tensor, t: int,
                   gamma: float, mode: int = B.MODE_TRIGGER, normalize: bool = True,
                   params: Optional[NSParams] = None, d: Optional[torch.Tensor] = None,
                   err: Optional[torch.Tensor] = None, refreshed: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None):
    """Returns (d, err, refreshed); q and cache_state are updated in place."""
    _dev(x, "x")
    batch, m, n = _bmn(x)
    r = min(m, n)
    if q.dtype != torch.float32 or q.numel() != batch * r * r:
        raise ValueError("q must be float32 [batch, r, r]")
    if cache_state.dtype != torch.int32 or cache_state.numel() != 2 * batch:
        raise ValueError("cache_state must be int32 [batch, 2]")
    _dev(q, "q"); _dev(cache_state, "cache_state")
    p = params or NSParams()
    d = torch.empty_like(x) if d is None else d
    err = torch.empty(batch, dtype=torch.float32, device=x.device) if err is None else err
    refreshed = (torch.empty(batch, dtype=torch.int32, device=x.device)
                 if refreshed is None else refreshed)
    _expect(d, "d", x.shape, x.dtype)
    _expect(err, "err", dtype=torch.float32, min_numel=batch)
    _expect(refreshed, "refreshed", dtype=torch.int32, min_numel=batch)
    ws = _ws(gram_ns_cached_ws(x.dtype, batch, m, n), x.device, ws)
    cp = p.c_struct()
    code = B.lib().sm_gram_ns_cached(x.data_ptr(), d.data_ptr(), q.data_ptr(),
                                     cache_state.data_ptr(), err.data_ptr(),
                                     refreshed.data_ptr(), _dt(x), batch, m, n, int(normalize),
                                     ctypes.byref(cp), gamma, mode, t, ws.data_ptr(),
                                     ws.numel() * ws.element_size(), _stream())
    B.check(code, "sm_gram_ns_cached")
    return d, err, refreshed


# ------------------------------------------------------------------ sign / vote

def sign_pack(x: torch.Tensor, bits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Packed signs as an int64 tensor holding the uint64 words."""
    _dev(x, "x")
    count = x.numel()
    words = (count + 63) // 64
    bits = torch.empty(max(words, 1), dtype=torch.int64, device=x.device) if bits is None else bits
    _expect(bits, "bits", dtype=torch.int64, min_numel=words)
    code = B.lib().sm_sign_pack(x.data_ptr(), _dt(x), count, bits.data_ptr(), _stream())
    B.check(code, "sm_sign_pack")
    return bits


def vote_update(bits: torch.Tensor, w: torch.Tensor, lr: float,
                vote_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bits: int64 [M, words_stride]; w updated in place; returns w."""
    _dev(bits, "bits"); _dev(w, "w")
    if bits.dtype != torch.int64 or bits.dim() != 2:
        raise ValueError("bits must be int64 [M, words_stride]")
    M, stride = bits.shape
    if stride * 64 < w.numel():
        raise ValueError("bits rows hold fewer than w.numel() signs")
    vp = 0
    if vote_out is not None:
        _dev(vote_out, "vote_out")
        if vote_out.dtype != torch.int8 or vote_out.numel() != w.numel():
            raise ValueError("vote_out must be int8 with w's element count")
        vp = vote_out.data_ptr()
    code = B.lib().sm_vote_update(bits.data_ptr(), M, stride, w.numel(), w.data_ptr(), _dt(w),
                                  lr, vp, _stream())
    B.check(code, "sm_vote_update")
    return w


def sign_int8(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 signs (-1 iff x < 0, else +1) of x's elements, flat [numel]."""
    _dev(x, "x")
    out = torch.empty(x.numel(), dtype=torch.int8, device=x.device) if out is None else out
    if out.dtype != torch.int8 or out.numel() < x.numel():
        raise ValueError("out must be int8 with at least x.numel() elements")
    code = B.lib().sm_sign_int8(x.data_ptr(), _dt(x), x.numel(), out.data_ptr(), _stream())
    B.check(code, "sm_sign_int8")
    return out


def vote_update_int8(signs: torch.Tensor, w: torch.Tensor, lr: float,
                     vote_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """signs: int8 [M, stride] (stride >= w.numel()); w updated in place; returns w."""
    _dev(signs, "signs"); _dev(w, "w")
    if signs.dtype != torch.int8 or signs.dim() != 2:
        raise ValueError("signs must be int8 [M, stride]")
    M, stride = signs.shape
    if stride < w.numel():
        raise ValueError("signs rows hold fewer than w.numel() signs")
    vp = 0
    if vote_out is not None:
        _dev(vote_out, "vote_out")
        if vote_out.dtype != torch.int8 or vote_out.numel() != w.numel():
            raise ValueError("vote_out must be int8 with w's element count")
        vp = vote_out.data_ptr()
    code = B.lib().sm_vote_update_int8(signs.data_ptr(), M, stride, w.numel(), w.data_ptr(),
                                       _dt(w), lr, vp, _stream())
    B.check(code, "sm_vote_update_int8")
    return w


def vote(signs: torch.Tensor, count: int, out: torch.Tensor) -> torch.Tensor:
    """The vote V in {-1, 0, +1} written to out ([count] float32/bfloat16).
    signs: int64 [M, words_stride] packed bits, or int8 [M, stride] signs."""
    _dev(signs, "signs"); _dev(out, "out")
    if signs.dim() != 2 or signs.dtype not in (torch.int64, torch.int8):
        raise ValueError("signs must be int64 (packed bits) or int8, shape [M, stride]")
    enc = B.ENC_BITS if signs.dtype == torch.int64 else B.ENC_INT8
    M, stride = signs.shape
    if out.numel() < count:
        raise ValueError("out is smaller than count")
    if stride * (64 if enc == B.ENC_BITS else 1) < count:
        raise ValueError("signs rows hold fewer than count signs")
    code = B.lib().sm_vote(signs.data_ptr(), enc, M, stride, count, out.data_ptr(), _dt(out),
                           _stream())
    B.check(code, "sm_vote")
    return out


def polar_update(w: torch.Tensor, d: torch.Tensor, lr: float) -> torch.Tensor:
    """w <- rnd(w - lr * d) in place (d has w's element count); returns w."""
    _dev(w, "w"); _dev(d, "d")
    if d.numel() != w.numel():
        raise ValueError("d must have w's element count")
    code = B.lib().sm_polar_update(w.data_ptr(), _dt(w), d.data_ptr(), _dt(d), w.numel(), lr,
                                   _stream())
    B.check(code, "sm_polar_update")
    return w


def spectral_norm(a: torch.Tensor, b: Optional[torch.Tensor], v0: torch.Tensor,
                  iters: int, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Power-method ||a - b||_2 per problem (b None: ||a||_2).

    a, b: [batch, m, n] or [m, n] (same dtype); v0: float32 [batch, n] start
    vectors.  Returns float32 [batch]."""
    _dev(a, "a"); _dev(v0, "v0")
    batch, m, n = _bmn(a)
    if b is not None:
        _dev(b, "b")
        if b.shape != a.shape or b.dtype != a.dtype:
            raise ValueError("b must match a in shape and dtype")
    if v0.dtype != torch.float32 or v0.numel() != batch * n:
        raise ValueError("v0 must be float32 with batch * n entries")
    out = torch.empty(batch, dtype=torch.float32, device=a.device)
    need = ctypes.c_size_t(0)
    B.check(B.lib().sm_spectral_norm_ws(batch, m, n, ctypes.byref(need)), "sm_spectral_norm_ws")
    ws = _ws(need.value, a.device, ws)
    code = B.lib().sm_spectral_norm(a.data_ptr(), b.data_ptr() if b is not None else None,
                                    _dt(a), batch, m, n, v0.data_ptr(), iters, out.data_ptr(),
                                    ws.data_ptr(), ws.numel() * ws.element_size(), _stream())
    B.check(code, "sm_spectral_norm")
    return out


# ------------------------------------------------------------------ sm_step

@dataclass
class MatrixBuffers:
    """Caller-owned state of one weight matrix (all on the GPU)."""
    w: torch.Tensor                       # [m, n]
    mom: torch.Tensor                     # [M, m, n]
    grad: torch.Tensor                    # [M, m, n]
    q_cache: Optional[torch.Tensor] = None      # [M, r, r] float32 (CacheMuon)
    cache_state: Optional[torch.Tensor] = None  # [M, 2] int32 (CacheMuon)

    def c_struct(self) -> B.Matrix:
        m, n = self.w.shape
        return B.Matrix(m, n, self.w.data_ptr(), self.mom.data_ptr(), self.grad.data_ptr(),
                        self.q_cache.data_ptr() if self.q_cache is not None else None,
                        self.cache_state.data_ptr() if self.cache_state is not None else None)


def _check_mats(cfg: StepConfig, mats: Sequence[MatrixBuffers], diag: Optional[torch.Tensor]):
    """Every tensor of every matrix has the shape and dtype the configuration
    implies (the library reads and writes them through raw pointers), and
    is a contiguous GPU tensor."""
    if len(mats) == 0:
        raise ValueError("a step needs at least one matrix")
    tensors = []
    for j, mb in enumerate(mats):
        if mb.w.dim() != 2:
            raise ValueError(f"matrix {j}: w must be [m, n]")
        m, n = mb.w.shape
        r = min(m, n)
        want = [(mb.w, "w", None, cfg.wdt), (mb.mom, "mom", (cfg.M, m, n), cfg.mdt),
                (mb.grad, "grad", (cfg.M, m, n), cfg.gdt)]
        if cfg.algo == B.CACHE_MUON:
            if mb.q_cache is None or mb.cache_state is None:
                raise ValueError(f"matrix {j}: CacheMuon needs q_cache and cache_state")
            want += [(mb.q_cache, "q_cache", (cfg.M, r, r), torch.float32),
                     (mb.cache_state, "cache_state", (cfg.M, 2), torch.int32)]
        for t, name, shape, dtype in want:
            _expect(t, f"matrix {j} {name}", shape, dtype, dev=False)
            tensors.append((t, f"matrix {j} {name}"))
    if diag is not None:
        _expect(diag, "diag", dtype=torch.float32, min_numel=len(mats) * cfg.M * 2, dev=False)
        tensors.append((diag, "diag"))
    for t, name in tensors:
        _dev(t, name)


def _mats_array(mats: Sequence[MatrixBuffers]):
    arr = (B.Matrix * len(mats))()
    for i, mb in enumerate(mats):
        arr[i] = mb.c_struct()
    return arr


def step_ws(cfg: StepConfig, mats: Sequence[MatrixBuffers]) -> int:
    out = ctypes.c_size_t(0)
    c = cfg.c_struct()
    arr = _mats_array(mats)
    B.check(B.lib().sm_step_ws(ctypes.byref(c), arr, len(mats), ctypes.byref(out)), "sm_step_ws")
    return out.value


class StepCall:
    """A prepared sm_step call: marshalled structs and a workspace, reusable per step."""

    def __init__(self, cfg: StepConfig, mats: Sequence[MatrixBuffers],
                 ws: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None):
        _check_mats(cfg, mats, diag)
        self.cfg = cfg
        self.mats = list(mats)
        self._c = cfg.c_struct()
        self._arr = _mats_array(self.mats)
        nbytes = step_ws(cfg, self.mats)
        self.ws = _ws(nbytes, self.mats[0].w.device, ws)
        self.diag = diag

    def __call__(self, t: int):
        code = B.lib().sm_step(ctypes.byref(self._c), self._arr, len(self.mats), t,
                               self.ws.data_ptr(), self.ws.numel() * self.ws.element_size(),
                               self.diag.data_ptr() if self.diag is not None else None,
                               _stream())
        B.check(code, "sm_step")


def step(cfg: StepConfig, mats: Sequence[MatrixBuffers], t: int,
         ws: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None):
    StepCall(cfg, mats, ws, diag)(t)


class StepGraph:
    """sm_step at step index t, recorded once as a HIP graph (sm_step_graph)
    and replayed on the current stream by each call (sm_graph_launch).

    The matrices' buffers, the workspace and diag are bound at recording and
    must stay in place while the graph lives.  A LionMuon step's type follows
    t: record one graph at a Muon step and one at a Lion step (they may share
    a workspace).  CacheMuon is not recordable (SmError SM_ERR_UNSUPPORTED).
    """

    def __init__(self, cfg: StepConfig, mats: Sequence[MatrixBuffers], t: int,
                 ws: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None):
        self._h = None
        self._call = StepCall(cfg, mats, ws, diag)   # holds the buffers and the workspace
        c = self._call
        h = ctypes.c_void_p()
        code = B.lib().sm_step_graph(ctypes.byref(c._c), c._arr, len(c.mats), t,
                                     c.ws.data_ptr(), c.ws.numel() * c.ws.element_size(),
                                     c.diag.data_ptr() if c.diag is not None else None,
                                     ctypes.byref(h))
        B.check(code, "sm_step_graph")
        self._h = h
        self.t = t

    @property
    def ws(self) -> torch.Tensor:
        return self._call.ws

    def __call__(self):
        if self._h is None:
            raise RuntimeError("StepGraph: replay after close()")
        B.check(B.lib().sm_graph_launch(self._h, _stream()), "sm_graph_launch")

    def close(self):
        """Destroys the graph once every replay enqueued so far has finished."""
        if self._h is not None:
            h, self._h = self._h, None
            torch.cuda.synchronize(self._call.ws.device)
            B.check(B.lib().sm_graph_destroy(h), "sm_graph_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ AdamW

STATE8_DTYPES = (torch.float8_e4m3fn, torch.float8_e5m2)   # first, second moment


def _state_blocks(count: int) -> int:
    return (count + B.STATE8_BLOCK - 1) // B.STATE8_BLOCK


def _stream_of(index: int) -> int:
    """The current stream of device `index`, whichever device is current."""
    return torch._C._cuda_getCurrentRawStream(index)


def _call_on(index: int, name: str, *args):
    """The library's function `name` with device `index` current."""
    fn = getattr(B.lib(), name)
    if torch._C._cuda_getDevice() == index:
        code = fn(*args)
    else:
        with torch.cuda.device(index):
            code = fn(*args)
    if code:
        B.check(code, name)


def _check_all(**wanted):
    """Each name=(tensor, shape, dtype): a contiguous GPU tensor of that shape
    and type, all on one device.  (The order of the checks is the messages'.)"""
    for name, (t, shape, dtype) in wanted.items():
        if t.dtype != dtype or t.shape != shape:
            _expect(t, name, shape, dtype, dev=False)
    device = None
    for name, (t, _, _) in wanted.items():
        _dev(t, name)
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{', '.join(wanted)} must be on one device")


@dataclass
class AdamWConfig:
    lr: float = 1e-3
    beta1: float = 0.9                # betas with 8-bit states: at most 0.99999
    beta2: float = 0.999
    eps: float = 1e-8
    rounding: int = B.ROUND_NEAREST   # of bf16 weights without a master
    seed: int = 0                     # of the stochastic rounding, 0 .. 2^64 - 1; one per set

    def c_struct(self) -> B.AdamWConfig:
        if not 0 <= self.seed < 1 << 64:
            raise ValueError("seed must be in 0 .. 2^64 - 1")
        return B.AdamWConfig(self.lr, self.beta1, self.beta2, self.eps, self.rounding, self.seed)


@dataclass
class ParamBuffers:
    """Caller-owned buffers of one parameter (all on the GPU, any shape).

    Without w, m and v the parameter only enters grad_norm (a Muon step's
    gradients)."""
    grad: torch.Tensor                    # [M, *shape], rows contiguous; M = 1: also [*shape]
    w: Optional[torch.Tensor] = None      # [*shape] float32 / bfloat16
    m: Optional[torch.Tensor] = None      # [*shape] float32, or float8_e4m3fn
    v: Optional[torch.Tensor] = None      # [*shape] float32, or float8_e5m2
    m_scale: Optional[torch.Tensor] = None   # float32 [ceil(count/256)] of 8-bit states
    v_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None    # [*shape] float32 of bfloat16 weights
    weight_decay: float = 0.0
    lr_mult: float = 1.0

    @classmethod
    def with_state(cls, w: torch.Tensor, grad: torch.Tensor, fp8: bool = False,
                   master: bool = False, weight_decay: float = 0.0,
                   lr_mult: float = 1.0) -> "ParamBuffers":
        """The buffers of w before its first step: zero moments (8-bit ones with
        fp8), and a float32 copy of w with master."""
        def zeros(dtype):
            size = 4 if dtype == torch.float32 else 1
            return torch.zeros(w.numel() * size, dtype=torch.uint8,
                               device=w.device).view(dtype).view(w.shape)
        m, v = (zeros(d) for d in (STATE8_DTYPES if fp8 else (torch.float32,) * 2))
        ms, vs = ((torch.zeros(_state_blocks(w.numel()), device=w.device) for _ in range(2))
                  if fp8 else (None, None))
        return cls(grad=grad, w=w, m=m, v=v, m_scale=ms, v_scale=vs,
                   master=w.detach().float() if master else None, weight_decay=weight_decay,
                   lr_mult=lr_mult)

    def c_struct(self, M: int) -> B.Param:
        g, w = self.grad, self.w
        if w is None:
            count = g.numel() // M
            return B.Param(count, g.stride(0) if M > 1 else count, None, None, g.data_ptr(), None,
                           None, None, None, B.F32, _DT[g.dtype], B.STATE_F32, 0.0, 1.0)
        count = w.numel()
        fp8 = self.m_scale is not None
        return B.Param(count, g.stride(0) if M > 1 else count, w.data_ptr(),
                       self.master.data_ptr() if self.master is not None else None, g.data_ptr(),
                       self.m.data_ptr(), self.v.data_ptr(),
                       self.m_scale.data_ptr() if fp8 else None,
                       self.v_scale.data_ptr() if fp8 else None, _DT[w.dtype], _DT[g.dtype],
                       B.STATE_FP8 if fp8 else B.STATE_F32, self.weight_decay, self.lr_mult)


def _check_param(j: int, p: ParamBuffers, M: int, device):
    """The shapes and dtypes of one parameter agree, and every tensor is a
    contiguous GPU tensor (the gradient: every worker's row) on `device`."""
    def expect(name, shape, dtype=None):
        _expect(getattr(p, name), f"parameter {j} {name}", shape, dtype, dev=False)

    def some_dt(t, name):
        if t.dtype not in _DT:
            raise ValueError(f"parameter {j} {name} must be float32 or bfloat16, got {t.dtype}")

    some_dt(p.grad, "grad")
    tensors = []
    if p.w is None:
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            if getattr(p, name) is not None:
                raise ValueError(f"parameter {j}: {name} without w")
        if M > 1 and (p.grad.dim() < 1 or p.grad.shape[0] != M):
            raise ValueError(f"parameter {j} grad must have {M} rows, got {tuple(p.grad.shape)}")
        rows = p.grad[0] if M > 1 else p.grad
    else:
        some_dt(p.w, "w")
        shape = tuple(p.w.shape)
        if tuple(p.grad.shape) != (M, *shape) and not (M == 1 and tuple(p.grad.shape) == shape):
            raise ValueError(f"parameter {j} grad must have shape {(M, *shape)}, "
                             f"got {tuple(p.grad.shape)}")
        rows = p.grad[0] if tuple(p.grad.shape) != shape else p.grad
        if p.m is None or p.v is None:
            raise ValueError(f"parameter {j}: w needs m and v")
        if p.m.dtype == torch.float32:
            dts = (torch.float32, torch.float32)
            if p.m_scale is not None or p.v_scale is not None:
                raise ValueError(f"parameter {j}: float32 states have no scales")
        else:
            dts = STATE8_DTYPES
            if p.m_scale is None or p.v_scale is None:
                raise ValueError(f"parameter {j}: 8-bit states need m_scale and v_scale")
            for name in ("m_scale", "v_scale"):
                expect(name, (_state_blocks(p.w.numel()),), torch.float32)
                tensors.append((getattr(p, name), name))
        expect("m", shape, dts[0])
        expect("v", shape, dts[1])
        tensors += [(p.w, "w"), (p.m, "m"), (p.v, "v")]
        if p.master is not None:
            if p.w.dtype != torch.bfloat16:
                raise ValueError(f"parameter {j}: only bfloat16 weights have a master")
            expect("master", shape, torch.float32)
            tensors.append((p.master, "master"))
    tensors.append((rows, "grad"))
    for t, name in tensors:
        _dev(t, f"parameter {j} {name}")
    if any(t.device != device for t, _ in tensors):
        raise ValueError("all tensors of a set must be on one device")


def _plain(p: ParamBuffers, M: int, device) -> bool:
    """The common case at a glance: one worker's gradient, float32 states, all
    that _check_param asks for (290 parameters: a set in 1.1 ms, not 1.9)."""
    w, g, m, v = p.w, p.grad, p.m, p.v
    if M != 1 or w is None or m is None or v is None or p.master is not None or \
            p.m_scale is not None or p.v_scale is not None:
        return False
    shape, gshape, f32 = w.shape, g.shape, torch.float32
    return (w.dtype in _DT and g.dtype in _DT and m.dtype == f32 and v.dtype == f32 and
            m.shape == shape and v.shape == shape and
            (gshape == shape or (len(gshape) == len(shape) + 1 and gshape[0] == 1 and
                                 gshape[1:] == shape)) and
            w.is_contiguous() and g.is_contiguous() and m.is_contiguous() and v.is_contiguous() and
            w.device == device and g.device == device and m.device == device and
            v.device == device)


# Sets whose calls some graph has captured.  A graph holds the addresses of a
# set's tables and buffers, and no references: the set stays until its close().
_captured_sets = set()


def _capturing(index: int) -> bool:
    """Device `index`'s current stream is being captured into a graph."""
    if torch._C._cuda_getDevice() == index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


class ParamSet:
    """A list of parameters that one call works on (sm_param_set): its tables
    on the GPU, made once.

    The buffers are bound at construction (a ParamBuffers changed afterwards
    changes nothing in the set) and must stay in place while the set, or a
    graph captured from its calls, lives.  A set whose calls were
    captured is kept, with its buffers and workspace, until its close() is
    called, which has to wait until those graphs are replayed no more.  Calls
    on one set (steps and norms) must be ordered."""

    def __init__(self, params: Sequence[ParamBuffers], M: int = 1,
                 ws: Optional[torch.Tensor] = None):
        self._h = None
        if len(params) == 0:
            raise ValueError("a set needs at least one parameter")
        if M < 1:
            raise ValueError("M must be at least 1")
        self.params = list(params)
        # the tensors themselves: a field of a ParamBuffers may be set anew
        self._tensors = [(p.grad, p.w, p.m, p.v, p.m_scale, p.v_scale, p.master)
                         for p in self.params]
        self.M = M
        self.device = self.params[0].grad.device
        for j, p in enumerate(self.params):
            if not (self.device.type == "cuda" and _plain(p, M, self.device)):
                _check_param(j, p, M, self.device)
        arr = (B.Param * len(self.params))(*[p.c_struct(M) for p in self.params])
        need = ctypes.c_size_t(0)
        B.check(B.lib().sm_param_set_ws(arr, len(self.params), ctypes.byref(need)),
                "sm_param_set_ws")
        if ws is not None:
            _dev(ws, "ws")
            if ws.device != self.device:
                raise ValueError("ws must be on the tensors' device")
        self.ws = _ws(need.value, self.device, ws)
        self._index = self.device.index
        self._stream = _stream_of(self._index)   # which the tables' memory belongs to
        h = ctypes.c_void_p()
        _call_on(self._index, "sm_param_set_create", arr, len(self.params), M,
                 self.ws.data_ptr(), self.ws.numel() * self.ws.element_size(), self._stream,
                 ctypes.byref(h))
        self._h = h

    def _use(self) -> int:
        """The device's current stream, which the tables outlive the work on."""
        if self._h is None:
            raise RuntimeError("ParamSet: use after close()")
        s = _stream_of(self._index)
        if s != self._stream:
            self.ws.record_stream(torch.cuda.current_stream(self.device))
        if s and _capturing(self._index):   # the null stream cannot be captured
            _captured_sets.add(self)
        return s

    def close(self):
        """Ends the set, once no graph captured from its calls is replayed any more."""
        _captured_sets.discard(self)
        if self._h is not None:
            h, self._h = self._h, None
            B.lib().sm_param_set_destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _scalar(t: Optional[torch.Tensor], name: str, dtype, device):
    if t is None:
        return None
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one element, has {t.numel()}")
    if t.dtype != dtype or t.device != device:
        _expect(t, name, dtype=dtype)
        raise ValueError(f"{name} must be on the set's device")
    return t.data_ptr()


def adamw(cfg: AdamWConfig, pset: ParamSet, t: Optional[int] = None,
          step: Optional[torch.Tensor] = None, gscale: Optional[torch.Tensor] = None,
          lr_scale: Optional[torch.Tensor] = None):
    """One AdamW step over the set's parameters, in place.

    Either t (1-based) or step (int64 device tensor, the steps done so far,
    advanced by the call) gives the step's index.  gscale (grad_norm's second
    result) and lr_scale are float32 device scalars; a non-finite one skips
    the step."""
    if (t is None) == (step is None):
        raise ValueError("adamw needs t or step (one of them)")
    if t is not None and t < 1:
        raise ValueError("t must be at least 1")
    c = cfg.c_struct()
    dev = pset.device
    sp = _scalar(step, "step", torch.int64, dev)
    gp = _scalar(gscale, "gscale", torch.float32, dev)
    lp = _scalar(lr_scale, "lr_scale", torch.float32, dev)
    s = pset._use()
    _call_on(pset._index, "sm_adamw", ctypes.byref(c), pset._h, t or 0, sp, gp, lp, s)


def grad_norm(psets: Sequence[ParamSet], max_norm: float, scale: float = 1.0,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """float32 [2]: the global norm of the sets' (mean) gradients times |scale|,
    and the factor scale * min(1, max_norm / (norm + 1e-6)) for adamw's gscale
    (out[1:2]), NaN where the norm is not finite.  A Muon step takes no factor:
    its matrices are neither scaled nor skipped."""
    if len(psets) == 0:
        raise ValueError("grad_norm needs at least one set")
    first = psets[0]
    for p in psets:
        if p.device != first.device:
            raise ValueError("all sets must be on one device")
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=first.device)
    else:
        _expect(out, "out", (2,), torch.float32)
        if out.device != first.device:
            raise ValueError("out must be on the sets' device")
    for p in psets:
        s = p._use()
    arr = (ctypes.c_void_p * len(psets))(*[p._h for p in psets])
    _call_on(first._index, "sm_grad_norm", arr, len(psets), scale, max_norm, out.data_ptr(), s)
    return out


def state8_pack(m: torch.Tensor, v: torch.Tensor):
    """(m8, v8, m_scale, v_scale): 8-bit AdamW states of float32 ones, rounded
    to nearest.  m8 is float8_e4m3fn and v8 float8_e5m2, in m's shape; the
    scales are float32, one per 256 entries."""
    f32 = torch.float32
    _check_all(m=(m, m.shape, f32), v=(v, m.shape, f32))
    n, dev = m.numel(), m.device
    m8 = torch.empty_like(m, dtype=STATE8_DTYPES[0])
    v8 = torch.empty_like(m, dtype=STATE8_DTYPES[1])
    ms = torch.empty(_state_blocks(n), dtype=f32, device=dev)
    vs = torch.empty_like(ms)
    _call_on(dev.index, "sm_state8_pack", m.data_ptr(), v.data_ptr(), n, m8.data_ptr(),
             v8.data_ptr(), ms.data_ptr(), vs.data_ptr(), _stream_of(dev.index))
    return m8, v8, ms, vs


def state8_unpack(m8: torch.Tensor, v8: torch.Tensor, m_scale: torch.Tensor,
                  v_scale: torch.Tensor):
    """(m, v): the float32 values of 8-bit AdamW states, in m8's shape."""
    f32, n = torch.float32, m8.numel()
    blocks = (_state_blocks(n),)
    _check_all(m8=(m8, m8.shape, STATE8_DTYPES[0]), v8=(v8, m8.shape, STATE8_DTYPES[1]),
               m_scale=(m_scale, blocks, f32), v_scale=(v_scale, blocks, f32))
    m = torch.empty_like(m8, dtype=f32)
    v = torch.empty_like(m)
    index = m8.device.index
    _call_on(index, "sm_state8_unpack", m8.data_ptr(), v8.data_ptr(), m_scale.data_ptr(),
             v_scale.data_ptr(), n, m.data_ptr(), v.data_ptr(), _stream_of(index))
    return m, v


# ------------------------------------------------------------------ kernel accounting

def mfma_ceiling(out: torch.Tensor, blocks: int, iters: int, mode: int = 1,
                 src: Optional[torch.Tensor] = None) -> int:
    """Enqueue the MFMA ceiling probe (sm_mfma_ceiling) on the current stream;
    returns the flops it executes.  `out` is a float32 device tensor of at
    least blocks * 256 entries; mode 2 reads `src` (a device tensor whose
    byte size is a power of two from 64 KB to 64 MB)."""
    _expect(out, "out", dtype=torch.float32, min_numel=blocks * 256)
    sp, sb = None, 0
    if mode == 2:
        if src is None:
            raise ValueError("mode 2 needs a source buffer")
        _dev(src, "src")
        sp, sb = ctypes.c_void_p(src.data_ptr()), src.numel() * src.element_size()
    B.check(B.lib().sm_mfma_ceiling(int(mode), blocks, iters, sp, sb,
                                    ctypes.c_void_p(out.data_ptr()), _stream()),
            "sm_mfma_ceiling")
    return blocks * 4 * iters * 16 * 32768


def profile_enable(on: bool = True):
    B.check(B.lib().sm_profile_enable(int(on)), "sm_profile_enable")


def profile_reset():
    B.check(B.lib().sm_profile_reset(), "sm_profile_reset")


def profile_read(kind: str):
    """(total_ms, launches, algorithmic work) for one kernel kind; waits on its events."""
    k = B.KERNEL_KINDS.index(kind)
    ms, n, work = ctypes.c_double(0), ctypes.c_int64(0), ctypes.c_double(0)
    B.check(B.lib().sm_profile_read(k, ctypes.byref(ms), ctypes.byref(n), ctypes.byref(work)),
            "sm_profile_read")
    return ms.value, n.value, work.value


def profile_read_bytes(kind: str) -> float:
    """Algorithmic HBM bytes of one kernel kind (operands read once, outputs written once)."""
    k = B.KERNEL_KINDS.index(kind)
    b = ctypes.c_double(0)
    B.check(B.lib().sm_profile_read_bytes(k, ctypes.byref(b)), "sm_profile_read_bytes")
    return b.value
