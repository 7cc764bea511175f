"""Argument checks of the operators around the decode GEMV, on the CPU: every refusal comes back before the HIP
runtime is touched (fake device addresses, never dereferenced)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
A = P(0x1000)
OK, NULL, MISALIGNED, SHAPE, WORKSPACE, ARG = 0, 1, 2, 3, 4, 6
F32, F16, BF16 = 0, 1, 2
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    import memory_bound_decode_gemv_amd as m
    if not os.path.exists(m.LIB_PATH):
        from memory_bound_decode_gemv_amd import _build
        _build.build()
    return m.raw()


@pytest.mark.parametrize("args,expect", [
    ((A, A, A, 3, A, F32, A, 4, 64, 64, 1e-5), ARG),              # unknown type
    ((A, A, A, F32, A, -1, A, 4, 64, 64, 1e-5), ARG),
    ((A, A, A, F32, A, F32, A, 4, 64, 64, 0.0), ARG),             # eps
    ((A, A, A, F32, A, F32, A, 4, 64, 64, -1.0), ARG),
    ((A, A, A, F32, A, F32, A, 4, 64, 64, INF), ARG),
    ((A, A, A, F32, A, F32, A, 4, 64, 64, float("nan")), ARG),
    ((A, None, A, F32, A, F32, A, 4, 64, 64, 1e-5), ARG),         # a sum to store, without a residual
    ((A, A, A, F32, A, F32, A, -1, 64, 64, 1e-5), SHAPE),
    ((A, A, A, F32, A, F32, A, 1 << 31, 64, 64, 1e-5), SHAPE),
    ((A, A, A, F32, A, F32, A, 4, 48, 64, 1e-5), SHAPE),          # K % 32
    ((A, A, A, F32, A, F32, A, 4, 64, 63, 1e-5), SHAPE),          # ld < K
    ((A, A, A, F32, A, F32, A, 4, (1 << 26) + 32, 1 << 27, 1e-5), SHAPE),
    ((A, A, A, F32, A, F32, A, 4, 64, 1 << 31, 1e-5), SHAPE),
    ((None, A, A, F32, A, F32, A, 4, 64, 64, 1e-5), NULL),
    ((A, A, A, F32, None, F32, A, 4, 64, 64, 1e-5), NULL),
    ((A, A, A, F32, A, F32, None, 4, 64, 64, 1e-5), NULL),
    ((P(0x1002), A, A, F32, A, F32, A, 4, 64, 64, 1e-5), MISALIGNED),
    ((A, P(0x1001), A, F16, A, F32, A, 4, 64, 64, 1e-5), MISALIGNED),
    ((A, A, P(0x1001), BF16, A, F32, A, 4, 64, 64, 1e-5), MISALIGNED),
    ((A, A, A, F32, P(0x1002), F32, A, 4, 64, 64, 1e-5), MISALIGNED),
    ((A, A, A, F32, A, F32, P(0x1002), 4, 64, 64, 1e-5), MISALIGNED),
    ((None, None, None, F32, None, F32, None, 0, 64, 64, 1e-5), OK),
    ((None, None, None, F32, None, F32, None, 4, 0, 0, 1e-5), OK),
])
def test_rmsnorm_q8_1_rejects_before_launch(lib, args, expect):
    assert lib.dg_rmsnorm_q8_1(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    ((A, A, A, F32, A, F32, A, 3, 4, 63, 63, 63, 1e-5), ARG),      # Q8_1 is not a float output
    ((A, A, A, F32, A, F32, A, F32, 4, 63, 63, 62, 1e-5), SHAPE),  # ldy < K
    ((A, A, A, F32, A, F32, A, F32, 4, 63, 62, 63, 1e-5), SHAPE),
    ((A, A, A, F32, A, F32, P(0x1001), BF16, 4, 63, 63, 63, 1e-5), MISALIGNED),
    ((A, A, A, F32, A, F32, P(0x1002), F32, 4, 63, 63, 63, 1e-5), MISALIGNED),
    ((None, None, None, F32, None, F32, None, F32, 0, 63, 63, 63, 1e-5), OK),
])
def test_rmsnorm_rejects_before_launch(lib, args, expect):
    assert lib.dg_rmsnorm(*args, None) == expect


def test_binding_checks_operands():
    """Host tensors, other types, strided tensors and ones smaller than the call touches are refused."""
    import torch
    import memory_bound_decode_gemv_amd as dg
    t = torch.zeros(4, 64)
    for call in (lambda: dg.dg_rmsnorm(t, t[0], t), lambda: dg.dg_rmsnorm_q8_1(t, t[0], t),
                 lambda: dg.dg_sample_rows(t, t[0], t), lambda: dg.dg_gemv_q4_0_glu(t, t, t, t, 4, 256, 1)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        dg._dtype_id(torch.zeros(4, dtype=torch.int32), "x")
    assert [dg._dtype_id(torch.zeros(1, dtype=d), "x") for d in (torch.float32, torch.float16, torch.bfloat16)] == [0, 1, 2]
    assert dg._rows(t, "x", "M") == 4 and dg._rows(t[0], "x", "M") == 1
    for odd in (t.view(2, 2, 64), t[0, 0]):   # rows of one matrix only: nothing past the first is left out in silence
        with pytest.raises(ValueError, match="dimensions"):
            dg._rows(odd, "x", "M")
    host = t.get_device()   # -1: the checks of one operand, without a device
    assert dg._arg("x", t, host, torch.float32, 4 * 64 * 4) == t.data_ptr()
    assert dg._arg("x", None, host, torch.float32, 1000) is None
    with pytest.raises(ValueError, match="holds 1024 bytes but the call touches 1025"):
        dg._arg("x", t, host, torch.float32, 1025)
    with pytest.raises(TypeError, match="float32, expected torch.float16"):
        dg._arg("x", t, host, torch.float16, 0)
    with pytest.raises(ValueError, match="contiguous"):
        dg._arg("x", t[:, :5], host, torch.float32, 0)
    with pytest.raises(ValueError, match="host tensor"):
        dg._arg("x", t, 0, torch.float32, 0)


@pytest.mark.parametrize("args,expect", [
    ((A, 3, A, A, A, A, A, A, 4, 100, 100, None, 0), ARG),
    ((A, F32, A, A, A, A, A, A, -1, 100, 100, None, 0), SHAPE),
    ((A, F32, A, A, A, A, A, A, 1 << 31, 100, 100, None, 0), SHAPE),
    ((A, F32, A, A, A, A, A, A, 4, 0, 100, None, 0), SHAPE),
    ((A, F32, A, A, A, A, A, A, 4, (1 << 31) - 1, 1 << 31, A, 1 << 40), SHAPE),
    ((A, F32, A, A, A, A, A, A, 4, 100, 99, None, 0), SHAPE),
    ((None, F32, A, A, A, A, A, A, 4, 100, 100, None, 0), NULL),
    ((A, F32, None, A, A, A, A, A, 4, 100, 100, None, 0), NULL),
    ((A, F32, A, A, A, A, A, None, 4, 100, 100, None, 0), NULL),
    ((P(0x1002), F32, A, A, A, A, A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((P(0x1001), BF16, A, A, A, A, A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, P(0x1002), A, A, A, A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, P(0x1002), A, A, A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, A, P(0x1002), A, A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, A, A, P(0x1002), A, A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, A, A, A, P(0x1002), A, 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, A, A, A, A, P(0x1004), 4, 100, 100, None, 0), MISALIGNED),
    ((A, F32, A, A, A, A, A, A, 4, 5000, 5000, None, 1 << 30), WORKSPACE),
    ((A, F32, A, A, A, A, A, A, 4, 5000, 5000, A, 1000), WORKSPACE),
    ((A, F32, A, A, A, A, A, A, 4, 5000, 5000, P(0x1004), 1 << 30), MISALIGNED),
    ((None, F32, None, None, None, None, None, None, 0, 100, 100, None, 0), OK),
])
def test_sample_rows_rejects_before_launch(lib, args, expect):
    assert lib.dg_sample_rows(*args, None) == expect


def test_sample_workspace(lib):
    f = lib.dg_sample_workspace_bytes
    assert f(0, 128256) == 0 and f(-1, 128256) == 0 and f(7, 4096) == 0
    one = f(1, 4097)
    assert one > 0 and f(3, 128256) == 3 * one and f(512, 4097) == 512 * one == f(100000, 4097)


@pytest.mark.parametrize("args,expect", [
    ((A, A, A, A, 4, 256, 1, 4), ARG),                # unknown activation
    ((A, A, A, A, 4, 256, 1, -1), ARG),
    ((A, A, A, A, 4, 100, 1, 0), SHAPE),              # K % 256
    ((A, A, A, A, 4, 256, 25, 0), SHAPE),
    ((A, A, A, A, 4, 256, -1, 0), SHAPE),
    ((A, A, A, A, -1, 256, 1, 0), SHAPE),
    ((A, A, A, A, 1 << 31, 256, 1, 0), SHAPE),
    ((A, A, A, A, 4, (1 << 26) + 256, 1, 0), SHAPE),
    ((None, A, A, A, 4, 256, 1, 0), NULL),
    ((A, None, A, A, 4, 256, 1, 0), NULL),
    ((A, A, None, A, 4, 256, 1, 0), NULL),
    ((A, A, A, None, 4, 256, 1, 0), NULL),
    ((P(0x1008), A, A, A, 4, 256, 1, 0), MISALIGNED),
    ((A, P(0x1008), A, A, 4, 256, 1, 0), MISALIGNED),
    ((A, A, P(0x1004), A, 4, 256, 1, 0), MISALIGNED),
    ((A, A, A, P(0x1002), 4, 256, 1, 0), MISALIGNED),
    ((None, None, None, None, 0, 256, 1, 0), OK),
    ((None, None, None, None, 4, 256, 0, 0), OK),
])
def test_gemv_glu_rejects_before_launch(lib, args, expect):
    for f in ("q4_0", "q8_0"):
        assert getattr(lib, f"dg_gemv_{f}_glu")(*args, None) == expect
        assert getattr(lib, f"dg_gemv_{f}_tiles_glu")(*args, None) == expect

