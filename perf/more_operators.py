"""The feed-forward layers' operators on real work: the cases, their inputs and their plain forms.

The gradients that the Muon and AdamW steps read come out of feed-forward
layers: a linear one, y = act(x W^T + bias) + residual, and a gated one,
h = act(x Wg^T) * (x Wu^T).  A training pass keeps a layer's input, in 8 bits
if it is to save memory, and the backward pass makes the activation again
from it and writes the weights' gradients into a worker's gradient stream,
or adds them to it.

8-bit checkpoints: 32 consecutive entries of a row share a power of two as
their scale, the smallest one (at least 2^-117) that brings the largest
magnitude to at most 448, the largest code of e4m3; codes are rounded to
nearest even.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ---------------------------------------------------------------- cases

def listed():
    block = {"d": 4096, "n": 11008, "dt": "bf16", "act": "silu"}
    return [
        # A short odd input kept in 8 bits: latency, blocks cut short.
        {"name": "act8 pack odd", "op": "pack", "T": 77, "d": 1283, "dt": "f32"},
        # The input of a feed-forward block of the LionMuon benchmark, for 8192 tokens.
        {"name": "act8 pack blocks", "op": "pack", "T": 8192, "d": 4096, "dt": "bf16"},
        # The inner activations of the same block, to be looked at or used elsewhere.
        {"name": "act8 unpack blocks", "op": "unpack", "T": 8192, "d": 11008, "dt": "bf16"},
        # One new token through the block's down projection, onto the residual stream: the weights' bytes.
        {"name": "linear token", "op": "linear", "T": 1, "d": 11008, "n": 4096, "dt": "bf16",
         "act": "none", "bias": False, "residual": True},
        # The first product of GPT-2 large's feed-forward part, bias and activation in the epilogue.
        {"name": "linear gpt2 large", "op": "linear", "T": 4096, "d": 1280, "n": 5120, "dt": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False},
        # A small float32 layer of odd sizes, backward: every tile is cut.
        {"name": "linear grad odd", "op": "linear_grad", "T": 515, "d": 771, "n": 1283, "dt": "f32",
         "act": "gelu", "bias": True, "kept": False, "add": True},
        # The down projection's backward from an 8-bit checkpoint of the inner activations.
        {"name": "linear grad down", "op": "linear_grad", "T": 8192, "d": 11008, "n": 4096, "dt": "bf16",
         "act": "none", "bias": False, "kept": True, "add": False},
        # One new token through the gated block: latency and the weights' bytes.
        {"name": "gated token", "op": "gated", "T": 1, **block},
        # A few tokens at once, as in speculative or batched generation.
        {"name": "gated batch", "op": "gated", "T": 19, **block},
        # A training pass of 8192 tokens.
        {"name": "gated blocks", "op": "gated", "T": 8192, **block},
        # A packed batch of uneven length through a narrower block, added to a stream.
        {"name": "gated grad ragged", "op": "gated_grad", "T": 1003, "d": 1280, "n": 3416, "dt": "bf16",
         "act": "silu", "kept": False, "add": True},
        # The largest: the whole backward pass of the block from its 8-bit checkpoint.
        {"name": "gated grad blocks", "op": "gated_grad", "T": 8192, "kept": True, "add": False, **block},
    ]


def draw(rng):
    def spread(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["pack", "unpack", "linear", "linear", "linear_grad", "linear_grad",
                     "gated", "gated", "gated_grad", "gated_grad"])
    case = {"op": op, "dt": rng.choice(["f32", "bf16", "bf16", "bf16"])}
    if op in ("pack", "unpack"):
        case.update(T=spread(1, 8192), d=spread(17, 8192))
        return case
    T, d, n = spread(1, 8192), spread(33, 6000), spread(33, 11008)
    if rng.random() < 0.6:  # models' widths; the others are odd ones
        d, n = -(-d // 64) * 64, -(-n // 64) * 64
    if case["dt"] == "f32":
        T = max(1, min(T, int(2e10 / (d * n))))
    case.update(T=T, d=d, n=n, act=rng.choice(ACTS))
    # x as columns of a wider tensor
    case["pad"] = rng.choice([0, 0, 0, 8, 5])
    if op.startswith("linear"):
        case["bias"] = rng.random() < 0.5
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    if op.endswith("_grad"):
        case["kept"] = rng.random() < 0.5
        case["add"] = rng.random() < 0.3
    return case


def work(case):
    op, T, d = case["op"], case["T"], case["d"]
    size = {"f32": 4, "bf16": 2}[case["dt"]]
    codes = T * d + T * -(-d // BLOCK)
    if op in ("pack", "unpack"):
        return {"bytes": codes + size * T * d, "flops": T * d}
    n = case["n"]
    both = 2 if op.startswith("gated") else 1
    if op in ("linear", "gated"):
        more = (case.get("bias", False)) * n + (case.get("residual", False)) * T * n
        return {"bytes": size * (T * d + both * n * d + T * n + more), "flops": 2 * both * T * d * n}
    again = 0 if case["act"] == "none" and both == 1 else 1
    x = codes if case["kept"] else size * T * d
    weights = both * n * d + case.get("bias", False) * n
    more = size * (T * n + T * d + weights * (3 if case["add"] else 2))
    return {"bytes": x + more, "flops": (4 + 2 * again) * both * T * d * n}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, T, d, dt = case["op"], case["T"], case["d"], TYPES[case["dt"]]

    def normal(*shape, size=1.0):
        return size * torch.randn(shape, generator=gen, device=dev)

    # normalised activations: some channels stand out, tokens differ in size
    x = normal(T, d) * torch.exp(0.3 * normal(T, 1))
    x *= torch.where(torch.rand(d, generator=gen, device=dev) < 0.005, 12.0, 1.0)
    s = {"op": op, "dt": dt}
    if op == "unpack":
        s["x8"], s["scale"] = _pack(x)
        return s
    pad = case.get("pad", 0)
    if pad:
        wide = torch.zeros(T, d + pad, device=dev, dtype=dt)
        wide[:, :d] = x
        s["x"] = wide[:, :d]
    else:
        s["x"] = x.to(dt)
    if op == "pack":
        return s
    n = case["n"]
    s["act"] = case["act"]
    s["weights"] = [normal(n, d, size=d ** -0.5).to(dt) for _ in range(2 if op.startswith("gated") else 1)]
    s["bias"] = normal(n, size=0.1).to(dt) if case.get("bias") else None
    if op in ("linear", "gated"):
        s["residual"] = normal(T, n).to(dt) if case.get("residual") else None
        return s
    if case["kept"]:
        s["x8"], s["scale"] = _pack(s.pop("x").float())
    dy = normal(T, n, size=1e-3)
    dy *= torch.rand(T, 1, generator=gen, device=dev) < 0.9  # no loss at prompts and padding
    s["dy"] = dy.to(dt)
    s["add"] = case["add"]
    # a worker's gradient streams, of the weights and the bias
    given = s["weights"] + ([s["bias"]] if case.get("bias") else [])
    s["grads"] = [normal(*w.shape, size=1e-3).to(dt) for w in given]
    return s


# ---------------------------------------------------------------- the plain forms

def _pack(x):
    """e4m3 codes [T, d] and the blocks' scales [T, ceil(d / 32)] (as e8m0)."""
    T, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % BLOCK)).view(T, -1, BLOCK)
    bits = x.abs().amax(2, keepdim=True).view(torch.int32)
    e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=10)
    codes = (x * ((254 - e) << 23).view(torch.float32)).to(torch.float8_e4m3fn)
    return (codes.view(T, -1)[:, :d].contiguous(),
            e.view(T, -1).to(torch.uint8).view(torch.float8_e8m0fnu))


def _unpack(codes, scale):
    d = codes.shape[1]
    scale = (scale.view(torch.uint8).to(torch.int32) << 23).view(torch.float32)
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :d]


def _act(name, z):
    if name == "relu":
        return z * (z > 0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _linear(s):
    y = s["x"].float() @ s["weights"][0].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(s["act"], y)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["dt"])


def _gated(s):
    x, (wg, wu) = s["x"].float(), s["weights"]
    return (_act(s["act"], x @ wg.float().t()) * (x @ wu.float().t())).to(s["dt"])


def _grads(s):
    """The gradient of x, and the weights' (and the bias's) in the worker's streams."""
    x = _unpack(s["x8"], s["scale"]) if "x8" in s else s["x"].float()
    weights = [w.float() for w in s["weights"]]
    dy, act = s["dy"].float(), s["act"]
    if s["op"] == "gated_grad":
        a, b = x @ weights[0].t(), x @ weights[1].t()
        dz = [dy * b * _slope(act, a), dy * _act(act, a)]
    elif act == "none":
        dz = [dy]
    else:
        z = x @ weights[0].t()
        dz = [dy * _slope(act, z if s["bias"] is None else z + s["bias"].float())]
    dx = dz[0] @ weights[0]
    if len(dz) > 1:
        dx = dx + dz[1] @ weights[1]
    new = [g.t() @ x for g in dz] + ([dz[0].sum(0)] if s["bias"] is not None else [])
    for old, g in zip(s["grads"], new):
        old.copy_(old.float() + g if s["add"] else g)
    return [dx.to(s["dt"])] + s["grads"]


def run(state):
    s = state
    op = s["op"]
    if own:
        import matrix_aware_optimizer_momentum_amd as sm
        if op == "pack":
            kept = sm.act8_pack(s["x"])
            return [kept.codes, kept.scale]
        if op == "unpack":
            return sm.act8_unpack(sm.Act8(s["x8"], s["scale"]), s["dt"])
        act = {"none": sm.ACT_NONE, "relu": sm.ACT_RELU, "silu": sm.ACT_SILU, "gelu": sm.ACT_GELU,
               "gelu_tanh": sm.ACT_GELU_TANH}[s["act"]]
        if op == "linear":
            return sm.linear(s["x"], s["weights"][0], bias=s["bias"], act=act, residual=s["residual"])
        if op == "gated":
            return sm.gated(s["x"], *s["weights"], act=act)
        x = sm.Act8(s["x8"], s["scale"]) if "x8" in s else s["x"]
        if op == "gated_grad":
            return sm.gated_grad(s["dy"], x, *s["weights"], act=act, dwg=s["grads"][0], dwu=s["grads"][1],
                                 accumulate=s["add"])
        got = sm.linear_grad(s["dy"], x, s["weights"][0], bias=s["bias"], act=act, dw=s["grads"][0],
                             db=s["grads"][1] if s["bias"] is not None else None, accumulate=s["add"])
        return [g for g in got if g is not None]
    if op == "pack":
        return list(_pack(s["x"].float()))
    if op == "unpack":
        return _unpack(s["x8"], s["scale"]).to(s["dt"])
    return _linear(s) if op == "linear" else _gated(s) if op == "gated" else _grads(s)


# ---------------------------------------------------------------- in 64 bits

def _two(e):
    """2^e, made of its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _step(x):
    """2^e, e >= -117 the least with every |x| of the block at most 448 * 2^e (448 = 0.875 * 2^9)."""
    f, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    k = torch.where(f > 0.875, e - 8, e - 9).clamp(min=-117)
    return _two(torch.where(f == 0, -117, k))


def _values(codes, scale):
    e = scale.view(torch.uint8).long() - 127
    return codes.double() * _two(e).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _both(name, z):
    """The activation and its derivative, through the error function's complement and the logistic function."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * (-z * z / 2).exp() / math.sqrt(2 * math.pi)
    u, du = z, torch.ones_like(z)
    if name == "gelu_tanh":  # (1 + tanh(q)) / 2 is the logistic function of 2 q
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(u)
    return z * p, p + z * p * torch.sigmoid(-u) * du


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "pack":
        T, d = s["x"].shape
        x = torch.cat([s["x"].double(), s["x"].new_zeros(T, -d % BLOCK).double()], 1).view(T, -1, BLOCK)
        scale = _step(x)
        q = _two((torch.frexp(x / scale)[1] - 1).clamp(min=-6) - 3)
        codes = torch.round(x / scale / q) * q
        return [codes.view(T, -1)[:, :d], scale.view(T, -1)]
    x = _values(s["x8"], s["scale"]) if "x8" in s else s["x"].double()
    if op == "unpack":
        return x
    w = torch.cat(s["weights"]).double()
    n = s["weights"][0].shape[0]
    z = torch.mm(x, w.T)
    a, da = _both(s["act"], z[:, :n] if s["bias"] is None else z[:, :n] + s["bias"].double())
    if op == "gated":
        return a * z[:, n:]
    if op == "linear":
        return a if s["residual"] is None else a + s["residual"].double()
    dy = s["dy"].double()
    dz = torch.cat([dy * z[:, n:] * da, dy * a], 1) if op == "gated_grad" else dy * da
    dw = torch.mm(dz.T, x)
    new = [dw[:n], dw[n:]] if op == "gated_grad" else [dw]
    if s["bias"] is not None:
        new.append(dz.sum(0))
    if s["add"]:
        new = [g + old.double() for g, old in zip(new, s["grads"])]
    return [torch.mm(dz, w)] + new
