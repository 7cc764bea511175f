"""Argument checks of the operators whose rows have weights or state of their own, on the CPU: every refusal comes back
before the HIP runtime is touched (fake device addresses, never dereferenced)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
A = P(0x1000)
OK, NULL, MISALIGNED, SHAPE, WORKSPACE, ARG = 0, 1, 2, 3, 4, 6
F32, F16, BF16 = 0, 1, 2
INF, NAN = float("inf"), float("nan")
BIG = 1 << 40   # a workspace's size


@pytest.fixture(scope="module")
def lib():
    import memory_bound_decode_gemv_amd as m
    if not os.path.exists(m.LIB_PATH):
        from memory_bound_decode_gemv_amd import _build
        _build.build()
    return m.raw()


@pytest.mark.parametrize("args,expect", [
    ((A, 3, A, A, A, 4, 8, 8, 2, 0, 1, 1.0), ARG),               # unknown type
    ((A, F32, A, A, A, 4, 8, 8, 2, 2, 1, 1.0), ARG),             # unknown score
    ((A, F32, A, A, A, 4, 8, 8, 2, -1, 1, 1.0), ARG),
    ((A, F32, A, A, A, 4, 8, 8, 2, 0, 1, INF), ARG),
    ((A, F32, A, A, A, 4, 8, 8, 2, 0, 1, NAN), ARG),
    ((A, F32, A, A, A, -1, 8, 8, 2, 0, 1, 1.0), SHAPE),
    ((A, F32, A, A, A, 1 << 31, 8, 8, 2, 0, 1, 1.0), SHAPE),
    ((A, F32, A, A, A, 4, 0, 8, 2, 0, 1, 1.0), SHAPE),
    ((A, F32, A, A, A, 4, 1025, 1025, 2, 0, 1, 1.0), SHAPE),     # E > 1024
    ((A, F32, A, A, A, 4, 8, 7, 2, 0, 1, 1.0), SHAPE),           # ld < E
    ((A, F32, A, A, A, 4, 8, 1 << 31, 2, 0, 1, 1.0), SHAPE),
    ((A, F32, A, A, A, 4, 8, 8, 0, 0, 1, 1.0), SHAPE),           # k
    ((A, F32, A, A, A, 4, 8, 8, 9, 0, 1, 1.0), SHAPE),           # k > E
    ((A, F32, A, A, A, 4, 128, 128, 65, 0, 1, 1.0), SHAPE),      # k > 64
    ((None, F32, A, A, A, 4, 8, 8, 2, 0, 1, 1.0), NULL),
    ((A, F32, A, None, A, 4, 8, 8, 2, 0, 1, 1.0), NULL),
    ((A, F32, A, A, None, 4, 8, 8, 2, 0, 1, 1.0), NULL),
    ((P(0x1002), F32, A, A, A, 4, 8, 8, 2, 0, 1, 1.0), MISALIGNED),
    ((P(0x1001), BF16, A, A, A, 4, 8, 8, 2, 0, 1, 1.0), MISALIGNED),
    ((A, F32, P(0x1002), A, A, 4, 8, 8, 2, 0, 1, 1.0), MISALIGNED),
    ((A, F32, A, P(0x1002), A, 4, 8, 8, 2, 0, 1, 1.0), MISALIGNED),
    ((A, F32, A, A, P(0x1002), 4, 8, 8, 2, 0, 1, 1.0), MISALIGNED),
    ((None, F32, None, None, None, 0, 8, 8, 2, 0, 1, 1.0), OK),
])
def test_route_rejects_before_launch(lib, args, expect):
    assert lib.dg_moe_route(*args, None) == expect


def moe(**change):
    """Arguments of dg_moe_q4_0 and dg_moe_q8_0 with some changed."""
    v = dict(Wg=A, Wu=A, Wd=A, Xq=A, ids=A, weights=A, Y=A, ydtype=F32, N=512, K=256, M=3, E=8, k=2, act=0, ws=A, ws_bytes=BIG)
    assert set(change) <= set(v)
    return tuple((v | change).values())


NOTHING = dict(Wg=None, Wu=None, Wd=None, Xq=None, ids=None, weights=None, Y=None, ws=None, ws_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(act=4), ARG), (dict(act=-1), ARG), (dict(ydtype=3), ARG),
    (dict(N=500), SHAPE), (dict(K=128), SHAPE), (dict(N=-256), SHAPE), (dict(K=-256), SHAPE),
    (dict(N=(1 << 26) + 256), SHAPE), (dict(K=(1 << 26) + 256), SHAPE),
    (dict(M=-1), SHAPE), (dict(M=4097, k=1), SHAPE), (dict(M=2049), SHAPE), (dict(k=-1), SHAPE), (dict(k=4097, M=1), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(N=1 << 26, E=32), SHAPE),          # E * N
    (dict(K=1 << 26, E=32), SHAPE),
    *((dict([(n, None)]), NULL) for n in ("Wg", "Wu", "Wd", "Xq", "ids", "weights", "Y")),
    *((dict([(n, P(0x1008))]), MISALIGNED) for n in ("Wg", "Wu", "Wd", "Xq", "ws")),
    *((dict([(n, P(0x1002))]), MISALIGNED) for n in ("ids", "weights", "Y")),
    (dict(Y=P(0x1001), ydtype=BF16), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=6 * (16 * 36 + 256 * 4) - 1), WORKSPACE),
    (NOTHING | dict(M=0), OK), (NOTHING | dict(K=0), OK),
])
def test_moe_rejects_before_launch(lib, change, expect):
    assert lib.dg_moe_q4_0(*moe(**change), None) == expect
    assert lib.dg_moe_q8_0(*moe(**change), None) == expect


def test_workspace_sizes(lib):
    """Those that the documentation's layouts need, and none for shapes that are refused."""
    for N, K, M, k in ((256, 256, 1, 1), (14336, 4096, 32, 2), (768, 2048, 1, 8)):
        assert lib.dg_moe_workspace_bytes(N, K, M, k) >= M * k * (N // 32 * 36)
    assert lib.dg_moe_workspace_bytes(512, 256, 3, 0) == 0
    for N, K, M, k in ((255, 256, 1, 1), (256, 256, 4096, 2), (256, 256, -1, 1), (256, 256, 1, -1)):
        assert lib.dg_moe_workspace_bytes(N, K, M, k) == 0
    assert lib.dg_lora_workspace_bytes(3, 64, 8) >= 3 * 8 * 4
    for M, K, R in ((-1, 64, 8), (3, -8, 8), (3, (1 << 30) + 8, 8), (3, 64, 0), (3, 64, 520)):
        assert lib.dg_lora_workspace_bytes(M, K, R) == 0


def lora(**change):
    v = dict(x=A, dtype=F32, A=A, B=A, wdtype=F16, adapter=A, scale=A, ranks=A, base=A, Y=A, M=3, N=100, K=64, R=16, L=2,
             ld=64, ws=A, ws_bytes=BIG)
    assert set(change) <= set(v)
    return tuple((v | change).values())


@pytest.mark.parametrize("change,expect", [
    (dict(dtype=3), ARG), (dict(wdtype=F32), ARG), (dict(wdtype=-1), ARG),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(K=60), SHAPE), (dict(K=-8), SHAPE), (dict(K=(1 << 30) + 8, ld=(1 << 31) - 8), SHAPE), (dict(ld=56), SHAPE), (dict(ld=68), SHAPE), (dict(ld=1 << 31), SHAPE),
    (dict(R=0), SHAPE), (dict(R=12), SHAPE), (dict(R=520), SHAPE), (dict(L=-1), SHAPE), (dict(L=1 << 31), SHAPE),
    *((dict([(n, None)]), NULL) for n in ("x", "A", "B", "adapter", "Y")),
    *((dict([(n, P(0x1008))]), MISALIGNED) for n in ("x", "A", "B", "ws")),
    *((dict([(n, P(0x1002))]), MISALIGNED) for n in ("adapter", "scale", "ranks", "base", "Y")),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=3 * 16 * 4 - 1), WORKSPACE),
    (dict(x=None, A=None, B=None, adapter=None, Y=None, ws=None, M=0), OK),
    (dict(x=None, A=None, B=None, adapter=None, Y=None, ws=None, N=0), OK),
])
def test_lora_rejects_before_launch(lib, change, expect):
    assert lib.dg_lora_rows(*lora(**change), None) == expect


def adjustments(**change):
    import memory_bound_decode_gemv_amd as m
    v = dict(tokens=0x1000, lens=0x1000, prompt_lens=0x1000, T=10, ldt=10, repetition=0x1000, frequency=0x1000,
             presence=0x1000, bias_ids=0x1000, bias=0x1000, bias_lens=0x1000, B=4, mask=0x1000, ldm=4)
    assert set(change) <= set(v)
    return m.dg_adjustments(*(v | change).values())


B = P(0x2000)


@pytest.mark.parametrize("args,change,expect", [
    ((A, B, 3, 4, 100, 100, 100), {}, ARG),
    ((A, B, F32, 4, 100, 100, 100), dict(bias=None), ARG),
    ((A, B, F32, 4, 100, 100, 100), dict(bias_ids=None), ARG),
    ((A, B, F32, -1, 100, 100, 100), {}, SHAPE), ((A, B, F32, 1 << 31, 100, 100, 100), {}, SHAPE),
    ((A, B, F32, 4, -1, 100, 100), {}, SHAPE), ((A, B, F32, 4, (1 << 31) - 1, 1 << 31, 1 << 31), {}, SHAPE),
    ((A, B, F32, 4, 100, 99, 100), {}, SHAPE), ((A, B, F32, 4, 100, 100, 99), {}, SHAPE),
    ((A, B, F32, 4, 100, 1 << 31, 100), {}, SHAPE), ((A, B, F32, 4, 100, 100, 1 << 31), {}, SHAPE),
    ((A, A, F32, 4, 100, 100, 104), {}, SHAPE),          # in place, with other rows
    ((A, B, F32, 4, 100, 100, 100), dict(T=11), SHAPE), ((A, B, F32, 4, 100, 100, 100), dict(T=-1), SHAPE),
    ((A, B, F32, 4, 100, 100, 100), dict(ldt=1 << 31), SHAPE),
    ((A, B, F32, 4, 100, 100, 100), dict(T=(1 << 30) + 1, ldt=(1 << 31) - 1), SHAPE),
    ((A, B, F32, 4, 100, 100, 100), dict(B=-1), SHAPE), ((A, B, F32, 4, 100, 100, 100), dict(B=65536), SHAPE),
    ((A, B, F32, 4, 100, 100, 100), dict(ldm=3), SHAPE), ((A, B, F32, 4, 100, 100, 100), dict(ldm=1 << 31), SHAPE),
    ((None, B, F32, 4, 100, 100, 100), {}, NULL), ((A, None, F32, 4, 100, 100, 100), {}, NULL),
    ((P(0x1002), B, F32, 4, 100, 100, 100), {}, MISALIGNED), ((A, P(0x1001), F16, 4, 100, 100, 100), {}, MISALIGNED),
    *(((A, B, BF16, 4, 100, 100, 100), dict([(n, 0x1002)]), MISALIGNED) for n in
      ("tokens", "lens", "prompt_lens", "repetition", "frequency", "presence", "bias_ids", "bias", "bias_lens", "mask")),
    ((None, None, F32, 0, 100, 100, 100), {}, OK), ((None, None, F32, 4, 0, 100, 100), {}, OK),
])
def test_adjust_rejects_before_launch(lib, args, change, expect):
    assert lib.dg_adjust_rows(*args, adjustments(**change), None) == expect


def test_binding_checks_operands():
    """Host tensors, unknown names and wrong types are refused."""
    import torch
    import memory_bound_decode_gemv_amd as dg
    t, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: dg.dg_adjust_rows(t, t), lambda: dg.dg_moe_route(t, i, t),
                 lambda: dg.dg_moe_q4_0(t, t, t, t, i, t, t, 256, 256, 4, 2), lambda: dg.dg_lora_rows(t, t, t, i, t)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
