"""Assembly of the operators of a batch of different requests (CPU; hipcc only): what their results or their speed rest on."""
import os
import re

import pytest

from memory_bound_decode_gemv_amd import _build


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("batch")
    out = {}
    for name in ("moe.hip", "lora.hip", "adjust.hip"):
        path = str(d / (name + ".s"))
        _build.device_asm(os.path.join(_build.CSRC, name), path)
        out[name] = open(path).read()
    return out


def kernels(text, part):
    """(name, body) of the kernels whose mangled name holds `part`."""
    found = [(m.group(1), text[m.end():text.find(".Lfunc_end", m.end())]) for m in re.finditer(r"^(_Z\w+):", text, re.M)
             if part in m.group(1)]
    assert found, part
    return found


@pytest.mark.parametrize("part", ["k_moe_glu", "k_moe_down"])
def test_experts_products(asm, part):
    """Weights straight into registers with non-temporal 16-byte loads, sums on the int8 matrix cores, at most 128 registers
    a wave (16 waves to a CU), no atomics; columns of several tokens by LDS DMA."""
    t = asm["moe.hip"]
    for name, body in kernels(t, part):
        assert re.search(r"global_load_dwordx4 .* nt", body) and "v_mfma_i32_16x16x" in body
        assert "atomic" not in body and "scratch_" not in body and "v_accvgpr_read" not in body
        assert ("global_load_lds_dwordx4" in body) == ("down_tokens" not in name)
        regs = int(re.search(r"\.amdhsa_next_free_vgpr (\d+)", t[t.index(".amdhsa_kernel " + name):]).group(1))
        assert regs <= 128, (name, regs)


def test_experts_sum_and_single_tokens_round_every_step(asm):
    """The weighted sum is a product and an addition per slot, each rounded, in both kernels that make it: otherwise the
    number of tokens would change a token's result."""
    for part in ("k_moe_sum", "k_moe_down_tokens"):
        for _, body in kernels(asm["moe.hip"], part):
            tail = body[body.rindex("v_mfma"):] if "v_mfma" in body else body
            assert "v_add_f32" in tail and "v_mul_f32" in tail
    for _, body in kernels(asm["moe.hip"], "k_moe_sum"):
        assert not re.search(r"v_(fma|fmac|mad|mac)_(f32|mix)", body)


def test_router_in_registers(asm):
    """Maxima by lane moves, scores and sums in binary64, no LDS."""
    for _, body in kernels(asm["moe.hip"], "k_moe_route"):
        assert "ds_" not in body and "row_shr" in body and "row_bcast" in body and "_f64" in body


def test_adapters(asm):
    """16-byte loads, binary32 multiply-adds, no atomics; few LDS exchanges between lanes."""
    t = asm["lora.hip"]
    for _, body in kernels(t, "k_lora_"):
        assert "global_load_dwordx4" in body and "atomic" not in body and "v_dot2" not in body and "v_mfma" not in body
        assert re.search(r"v_(fma|fmac|fma_mix)_f32", body)   # mix: binary16 factors widened on the way
    for _, body in kernels(t, "k_lora_dots"):
        assert "ds_bpermute" not in body


def test_adjustments_round_every_step(asm):
    """No product fused into a sum or a conversion; counts by LDS additions of whole numbers, none in memory."""
    for _, body in kernels(asm["adjust.hip"], "k_adjust"):
        assert "v_fma_mix" not in body and "global_atomic" not in body and "flat_" not in body
        assert re.search(r"ds_(add|or)_rtn_u32|ds_(add|or)_rtn_b32", body)
