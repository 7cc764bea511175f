"""The kernels that the operators of a batch of different requests are built into are those that their launch rules can
choose, no others (CPU; hipcc only)."""
import os
import re

import pytest

from memory_bound_decode_gemv_amd import _build

BOTH = (0, 1)


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    d = tmp_path_factory.mktemp("built")

    def names(source):
        path = str(d / (source + ".s"))
        _build.device_asm(os.path.join(_build.CSRC, source), path)
        return re.findall(r"^\s*\.amdhsa_kernel (\w+)", open(path).read(), re.M)
    return {s: names(s) for s in ("moe.hip", "adjust.hip")}


def arguments(names, pattern):
    found = [m.groups() for m in (re.search(pattern, n) for n in names) if m]
    assert len(found) == len(set(found))
    return {tuple(int(v) if v.isdigit() else v for v in f) for f in found}


def test_gated_products(built):
    """Format, more than 8 columns, several row groups a workgroup, waves.  Several row groups go with rows of up to 2048
    of Q4_0 and eight waves with longer ones, so never together."""
    got = arguments(built["moe.hip"], r"k_moe_gluINS0_9Tiles(Q\d)_0ELb(\d)ELb(\d)ELi(\d)ELi2E")
    assert got == ({(f, many, 0, waves) for f in ("Q4", "Q8") for many in BOTH for waves in (4, 8)} |
                   {("Q4", many, 1, 4) for many in BOTH})


def test_down_products(built):
    """Format, more than 8 columns, several row groups a workgroup, parts of K: several row groups with one part alone."""
    got = arguments(built["moe.hip"], r"k_moe_downINS0_9Tiles(Q\d)_0ELb(\d)ELb(\d)ELi4ELi(\d)ELi2E")
    assert got == ({(f, many, 0, parts) for f in ("Q4", "Q8") for many in BOTH for parts in (1, 2)} |
                   {("Q4", many, 1, 1) for many in BOTH})


def test_adjustments(built):
    """Type, the table's words (j: 32 bits, t: 16), groups a thread.  32-bit words beside 16-bit logits stand for histories
    of more than 32767 tokens, whose list and table of four groups are 196 KiB of the 160 that there are."""
    got = arguments(built["adjust.hip"], r"k_adjustI(f|DF16_|DF16b)(j|t)Li(\d)E")
    assert got == ({("f", "j", g) for g in (1, 2, 4)} | {(e, "t", g) for e in ("DF16_", "DF16b") for g in (1, 2, 4)} |
                   {(e, "j", g) for e in ("DF16_", "DF16b") for g in (1, 2)})
