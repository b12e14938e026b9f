"""Properties of the generated gfx950 code of the AdamW kernels, checked on the
CPU from hipcc's assembly output (no GPU needed): no scratch, no flat memory
accesses (the tables' pointers are global memory), no packed float32
instructions, and the step's kernels within the registers of seven waves per
SIMD."""
import re
import subprocess
import os

import pytest

from matrix_aware_optimizer_momentum_amd import build_lib


@pytest.fixture(scope="module")
def adamw_asm(tmp_path_factory):
    try:
        hipcc = build_lib._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "k_adamw.s"
    src = os.path.join(build_lib.CSRC, "k_adamw.hip")
    proc = subprocess.run([hipcc, *build_lib.HIP_FLAGS, "--cuda-device-only", "-S", src, "-o",
                           str(out)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert proc.returncode == 0, proc.stdout[-2000:]
    return out.read_text()


def test_no_scratch_no_flat_accesses_no_packed_float32(adamw_asm):
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size\s+(\d+)", adamw_asm)
    assert len(sizes) >= 10 and all(int(v) == 0 for v in sizes)
    ops = re.findall(r"^\s+([a-z]\w+)", adamw_asm, re.M)
    assert not [o for o in ops if o.startswith(("flat_", "scratch_"))]
    assert not [o for o in ops if re.fullmatch(r"v_pk_(add|mul|fma)_f32", o)]


def test_the_step_leaves_registers_for_seven_waves(adamw_asm):
    found = re.findall(r"\.name:\s+(\S*k_adamwI\S*)\n(?:.*\n)*?\s+\.vgpr_count:\s+(\d+)", adamw_asm)
    assert len(found) == 2
    assert all(int(v) <= 72 for _, v in found), found


def test_codes_and_weights_are_made_by_the_hardware_conversions(adamw_asm):
    for op in ("v_cvt_scalef32_sr_fp8_f32", "v_cvt_scalef32_sr_bf8_f32", "v_cvt_sr_bf16_f32",
               "v_cvt_scalef32_pk_f32_fp8", "v_cvt_scalef32_pk_f32_bf8"):
        assert op in adamw_asm, op
