"""8-bit checkpoints of many blocks, where a workgroup takes four units of 64 of
them, on the GPU: codes, scales and values exactly as the definition gives."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_momentum_amd as sm
from oracle import layer_oracle as L
from tests.test_gpu_layer import DT, Guarded

pytestmark = pytest.mark.gpu


def two(e):
    """2^e in float64, made of its bits (a device's pow is not exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pack_reference(x):
    """(codes, scales) as uint8 of float32 x [T, d] on the CPU: act8_pack of the oracle, whole rows
    at a time."""
    T, d = x.shape
    nb = -(-d // L.BLOCK)
    v = torch.zeros(T, nb * L.BLOCK)
    v[:, :d] = x
    v = v.view(T, nb, L.BLOCK)
    fin = v.isfinite()
    mag = torch.where(fin, v.abs(), 0.0)
    f, e = np.frexp(mag.amax(2).numpy())   # 448 = 0.875 * 2^9
    e = np.where(f > 0.875, e - 8, e - 9)
    e = torch.from_numpy(np.where(f == 0, -117, np.maximum(e, -117)).astype(np.int32))
    q = torch.where(fin, v, 0.0).double() * two(-e)[..., None]
    q = torch.where((e == 120)[..., None], q.clamp(-240, 240), q)
    codes = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(fin, codes, torch.tensor(0x7F, dtype=torch.uint8))
    return codes.view(T, -1)[:, :d].contiguous(), (e + 127).to(torch.uint8)


def values_of(codes, scales, device):
    s = two(scales.to(device).long() - 127).repeat_interleave(L.BLOCK, 1)
    return codes.to(device).view(torch.float8_e4m3fn).float().double() * s[:, :codes.shape[1]]


# from 65536 blocks on a workgroup takes four units: rows of fewer than 256 blocks and of more,
# last blocks cut short, the last workgroup past the last row
MANY = [(8191, 1283), (70000, 31), (2049, 4100), (300, 8225)]


@pytest.mark.parametrize("layout", [(0, 0), (3, 5)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", MANY)
def test_act8_of_many_blocks(gpu_lib, T, d, dt, layout):
    assert T * -(-d // 32) >= 65536
    rng = np.random.default_rng(T)
    v = rng.standard_normal((T, d)) * np.exp(4 * rng.standard_normal((T, 1)))
    some = lambda share: rng.random((T, d)) < share
    v[some(0.1)] = 0.0
    for value in (np.inf, -np.inf, np.nan, 3.3e38, -3.3e38, 1e-38, 448.0):
        v[some(2e-4)] = value
    X = Guarded(v, dt, *layout)
    codes, scales = pack_reference(X.t.float().cpu())
    kept = sm.act8_pack(X.t)
    assert torch.equal(kept.scale.view(torch.uint8).cpu(), scales)
    assert torch.equal(kept.codes.view(torch.uint8).cpu(), codes)
    X.check("x")
    want = values_of(codes, scales, "cuda").nan_to_num(nan=-1.0)
    for to in DT:
        out = Guarded(np.zeros((T, d)), to, *layout)
        sm.act8_unpack(kept, DT[to], out=out.t)
        assert torch.equal(out.t.double().nan_to_num(nan=-1.0), want)
        out.check("values")


@pytest.mark.parametrize("to,T,d", [("f32", 8200, 8225), ("bf16", 8200, 16418)])
def test_values_past_the_caches(gpu_lib, to, T, d):
    """More than 256 MB of them: written past the caches."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    codes = torch.randint(0, 256, (T, d), generator=gen, device="cuda", dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.randint(10, 247, (T, -(-d // 32)), generator=gen, device="cuda", dtype=torch.uint8)
    assert T * d * DT[to].itemsize > 256 << 20
    got = sm.act8_unpack(sm.Act8(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)),
                         DT[to])
    for r in range(0, T, 1000):
        assert torch.equal(got[r:r + 1000].double(),
                           values_of(codes[r:r + 1000], scales[r:r + 1000], "cuda"))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(3000, 1283), (2100, 1024)])
def test_gradients_from_a_checkpoint_of_many_blocks(gpu_lib, T, d, dt):
    """Decoded into the call's workspace, rows of an odd length there with zeros behind them."""
    n = 40
    gen = torch.Generator().manual_seed(T)
    t = lambda *s: torch.randn(*s, generator=gen).to(DT[dt]).cuda()
    x, wg, wu, dy = t(T, d), t(n, d), t(n, d), t(T, n)
    kept = sm.act8_pack(x)
    values = sm.act8_unpack(kept, DT[dt])
    want = torch.tensor(L.act8_unpack(*(v.view(torch.uint8).cpu().numpy()
                                        for v in (kept.codes, kept.scale))))
    assert T * -(-d // 32) >= 65536 and torch.equal(values.double().cpu(), want)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")   # NaN
    for a, b in ((sm.gated_grad(dy, kept, wg, wu, ws=ws), sm.gated_grad(dy, values, wg, wu)),
                 (sm.linear_grad(dy, kept, wg, ws=ws), sm.linear_grad(dy, values, wg))):
        assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
