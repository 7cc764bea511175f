"""Assembly of the operators around the decode GEMV (CPU; hipcc only): what their results or their speed rest on."""
import os
import re

import pytest

from memory_bound_decode_gemv_amd import _build


def asm_of(name, tmp):
    out = str(tmp / (name + ".s"))
    _build.device_asm(os.path.join(_build.CSRC, name), out)
    return open(out).read()


def kernels(text, part):
    """Bodies of the kernels whose mangled name holds `part`."""
    found = [text[m.end():text.find(".Lfunc_end", m.end())] for m in re.finditer(r"^(_Z\w+):", text, re.M)
             if part in m.group(1)]
    assert found, part
    return found


def test_norm_rounds_twice_to_16_bits(tmp_path):
    """No sum or product is rounded to binary16 straight from its exact value, and the sums of squares are binary64."""
    t = asm_of("norm.hip", tmp_path)
    for body in kernels(t, "k_rmsnorm"):
        assert "v_fma_mix" not in body
        assert "v_fma_f64" in body or "v_fmac_f64" in body
        assert "ds_bpermute" not in body


def test_sampler_sums_whole_numbers(tmp_path):
    """Masses are added as 64-bit integers, in LDS and in memory; no floating-point atomics."""
    t = asm_of("sample.hip", tmp_path)
    for body in kernels(t, "k_sample_hist"):
        assert "ds_add_u64" in body and "global_atomic_add_x2" in body
    assert "atomic_add_f" not in t and "ds_add_f" not in t
    for body in kernels(t, "k_sample_"):
        assert "ds_bpermute" not in body


@pytest.mark.parametrize("name,part", [("gemv_tiles.hip", "k_glu_tiles")])
def test_tiled_gated_product(name, part, tmp_path):
    """Weights straight into registers with non-temporal 16-byte loads, columns by LDS DMA, sums on the matrix cores,
    no atomics and no scratch."""
    for body in kernels(asm_of(name, tmp_path), part):
        assert re.search(r"global_load_dwordx4 .* nt", body)
        assert "global_load_lds_dwordx4" in body and "v_mfma_i32_16x16x" in body
        assert "atomic" not in body and "scratch_" not in body and "v_accvgpr_read" not in body


def test_plain_units_kernels_pay_nothing_for_the_gated_form(tmp_path):
    """A wave of the units kernels stores 64 outputs at a time and the rest at the end: only the end depends on the
    lane.  The plain kernels take their own arguments (32 bytes, then the hidden ones) and no empty one."""
    t = asm_of("gemv_m1_units.hip", tmp_path)
    for body in kernels(t, "k_units"):
        assert body.count("s_and_saveexec_b64") == 1
    plain = [b for b in kernels(t, "k_units") if "GluArgs" not in b.split(".amdhsa_kernel", 1)[1].split("\n", 1)[0]]
    assert plain
    for body in plain:
        assert re.search(r"\.amdhsa_kernarg_size 288\b", body)


def test_norm_squares_and_sums_in_binary64(tmp_path):
    """Per element of a thread's groups one widening, one product and one addition in binary64, beside the ten additions
    over the workgroup.  (The root and the quotient are binary64 fused operations whatever the sum is.)"""
    t = asm_of("norm.hip", tmp_path)
    for groups in (0, 1, 2, 4):   # 0: rows read twice, a group at a time
        for body in kernels(t, f"ELi{groups}EEEvPKNT_"):
            n = 8 * max(groups, 1)
            assert body.count("v_cvt_f64_f32") >= n + 1   # and eps
            assert body.count("v_mul_f64") >= n and body.count("v_add_f64") >= n + 10
