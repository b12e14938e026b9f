"""Properties of the generated gfx950 code of the feed-forward layers' kernels,
checked on the CPU from hipcc's assembly output (no GPU needed): no scratch, no
packed float32 instructions, two waves to a SIMD, no product under a lane mask
without a skip, and the wait states around the direct-to-LDS loads, which their
inline assembly keeps out of the compiler's sight."""
import os
import re
import subprocess

import pytest

from matrix_aware_optimizer_momentum_amd import build_lib
from tests.test_kernel_code_cpu import _sgprs, masked_mfmas_without_skip

TILES = [f"k_layer_{t}_{m}" for t in ("bf16", "f32") for m in (4, 2, 1)]
UNITS = ["k_act8", "k_layer", "k_layer_few", *TILES]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    try:
        hipcc = build_lib._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    folder = tmp_path_factory.mktemp("asm")
    runs = []
    for u in UNITS:
        out = folder / f"{u}.s"
        runs.append((u, out, subprocess.Popen(
            [hipcc, *build_lib.HIP_FLAGS, "--cuda-device-only", "-S",
             os.path.join(build_lib.CSRC, u + ".hip"), "-o", str(out)],
            stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    texts = {}
    for u, out, p in runs:
        log = p.communicate()[0]
        assert p.returncode == 0, log[-2000:]
        texts[u] = out.read_text()
    return texts


def kernels(text):
    return {m.group(1): m.group(2) for m in
            re.finditer(r"^(_ZN2sm\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M)}


@pytest.mark.parametrize("unit", UNITS)
def test_no_scratch_and_no_packed_float32(asm, unit):
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size\s+(\d+)", asm[unit])
    assert sizes and all(int(v) == 0 for v in sizes)
    ops = re.findall(r"^\s+([a-z]\w+)", asm[unit], re.M)
    assert not [o for o in ops if o.startswith("scratch_")]
    assert not [o for o in ops if re.fullmatch(r"v_pk_(add|mul|fma)_f32", o)]


@pytest.mark.parametrize("unit", TILES)
def test_products_run_two_waves_to_a_simd(asm, unit):
    found = re.findall(r"\.name:\s+(\S*k_tile\S*)\n(?:.*\n)*?\s+\.vgpr_count:\s+(\d+)", asm[unit])
    assert len(found) == 6 and all(int(v) <= 256 for _, v in found), found
    bodies = {k: v for k, v in kernels(asm[unit]).items() if "k_tile" in k}
    assert len(bodies) == 6
    for name, body in bodies.items():
        assert not masked_mfmas_without_skip(body), name


def lds_load_hazards(body):
    """Direct-to-LDS buffer loads that read an SGPR which a VALU instruction wrote within the five
    instructions before (wait states: s_nop's argument + 1), or that follow an M0 write at once."""
    insts = [t for t in (line.split(";")[0].strip() for line in body.splitlines())
             if t and not t.endswith(":") and not t.startswith(".")]
    bad = []
    for n, t in enumerate(insts):
        if not (t.startswith("buffer_load") and t.endswith(" lds")):
            continue
        base = _sgprs(t.split(None, 1)[1].split(",")[1].strip())
        assert len(base) == 4, t
        dist = 0
        for back in range(n - 1, -1, -1):
            u = insts[back]
            if u.startswith("s_nop"):
                dist += int(u.split()[1], 0) + 1
                continue
            if back == n - 1 and re.match(r"s_mov_b32 m0,", u):
                bad.append((n, "M0 written just before", t))
            if u.startswith("v_") and " " in u and \
                    _sgprs(u.split(None, 1)[1].split(",")[0].strip()) & base and dist < 5:
                bad.append((n, u, t))
            dist += 1
            if dist >= 5:
                break
    return bad


@pytest.mark.parametrize("unit", TILES)
def test_wait_states_of_the_loads_into_lds(asm, unit):
    bodies = {k: v for k, v in kernels(asm[unit]).items() if "k_tile" in k}
    for name, body in bodies.items():
        assert body.count(" lds\n") >= 16, name
        assert not lds_load_hazards(body), name


def test_the_scan_finds_the_hazards():
    body = "\n".join(["\tv_readfirstlane_b32 s41, v7", "\ts_mov_b32 m0, s42", "\ts_nop 0",
                      "\tbuffer_load_dwordx4 v62, s[40:43], 0 offen lds",
                      "\tv_readfirstlane_b32 s40, v7", "\ts_nop 4", "\ts_mov_b32 m0, s42",
                      "\tbuffer_load_dwordx4 v61, s[40:43], 0 offen lds"])
    assert [b[0] for b in lds_load_hazards(body)] == [3, 7]


@pytest.mark.parametrize("unit", TILES)
def test_waves_that_share_a_simd(asm, unit):
    """By what the hardware holds: 512 VGPRs of a SIMD's lane (in eights), 160 KB of LDS of a CU,
    eight waves of a SIMD, four SIMDs."""
    mi = int(unit[-1])
    number = lambda entry, key: int(re.search(rf"\.{key}:\s+(\d+)", entry).group(1))
    found = [e for e in asm[unit].split("- .agpr_count:")[1:]
             if re.search(r"\.name:\s+\S*k_tile", e)]
    assert len(found) == 6
    for e in found:
        threads = number(e, "max_flat_workgroup_size")
        assert threads == 128 * mi
        by_lds = 163840 // number(e, "group_segment_fixed_size") * (threads // 64) // 4
        by_vgprs = 512 // (-(-number(e, "vgpr_count") // 8) * 8)
        assert min(by_lds, by_vgprs, 8) == (1 if mi == 1 else 2), e[:400]
