"""RMS norm with the residual's addition, into Q8_1 columns and float rows (GPU).

The definition fixes every rounding except the order of the binary64 sum of
squares, whose effect on r is below one binary32 rounding border in 10^8 rows,
so the bytes are compared exactly with a numpy statement of it (Q8_1 codes
through the oracle's quantiser).  The values are also compared with the norm
in 64 bits: r, h*r and (h*r)*w are each off by at most half a step.
"""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}   # smallest subnormal: an underflow's absolute step


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def draw(key, shape, dtype, std=1.0):
    """float32 values representable in dtype, on the host."""
    import torch
    v = torch.from_numpy(synth.normal_f32(key, shape, std))
    return v.to(tdtype(dtype))


def reference(x, res, w, eps=EPS):
    """(h in x's type, y float32, y in 64 bits) of CPU tensors."""
    import torch
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    h32 = h.float().numpy()
    w32 = w.float().numpy()
    h64 = h32.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        root = np.sqrt(np.mean(h64 * h64, axis=-1, keepdims=True) + np.float64(np.float32(eps)))
        r = (1.0 / root).astype(np.float32)
        y32 = (h32 * r) * w32
        y64 = h64 / root * w32.astype(np.float64)
    return h, y32, y64


def run_q8_1(dg, dev, x, res, w, K, ld, h_is=None, eps=EPS):
    import torch
    M = x.shape[0]
    xd, wd = x.to(dev), w.to(dev)
    rd = res.to(dev) if res is not None else None
    hd = None
    if rd is not None:
        hd = {"x": xd, "res": rd, "none": None}.get(h_is, torch.full((M, ld), 7.0, dtype=x.dtype, device=dev))
    Xq = torch.full((M * (K // 32) * 36 + 64,), 0xA5, dtype=torch.uint8, device=dev)
    dg.dg_rmsnorm_q8_1(xd, wd, Xq, res=rd, h=hd, eps=eps, M=M, K=K, ld=ld)
    torch.cuda.synchronize()
    got = Xq.cpu().numpy()
    assert (got[M * (K // 32) * 36:] == 0xA5).all(), "bytes behind the columns changed"
    return got[:M * (K // 32) * 36], (hd.cpu() if hd is not None else None)


# one group per thread, two, four, and rows that are read twice; quads at a wave's end
@pytest.mark.parametrize("K", [32, 64, 480, 2048, 4096, 8192, 8224, 16384, 32768, 32800, 70016])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_q8_1_bytes(dg, dev, orc, K, dtype):
    for M, with_res, wdtype in ((1, True, "f32"), (3, False, "bf16"), (5, True, "f16")):
        ld = K + (8 if M == 3 else 0)
        x = draw((1100, 1, M, K % 97), (M, ld), dtype, 1.7)
        res = draw((1101, 1, M, K % 97), (M, ld), dtype, 2.3) if with_res else None
        w = draw((1102, 1, M, K % 97), (K,), wdtype, 0.3)
        got, h = run_q8_1(dg, dev, x, res, w, K, ld)
        href, y32, _ = reference(x[:, :K], res[:, :K] if with_res else None, w)
        want = orc.quantize_q8_1(y32).reshape(-1)
        bad = np.flatnonzero(got != want)
        assert bad.size == 0, f"M={M} K={K}: {bad.size} bytes differ, first at {bad[0]}"
        if with_res:
            import torch
            assert torch.equal(h[:, :K].float(), href.float())
            assert (h[:, K:].float() == 7.0).all(), "columns behind K changed"


@pytest.mark.parametrize("K", [4096, 40000])   # in registers, and read a second time
@pytest.mark.parametrize("h_is", ["x", "res", "none"])
def test_residual_in_place(dg, dev, orc, K, h_is):
    import torch
    x, res = draw((1110, 1, 0, 0), (2, K), "bf16"), draw((1110, 1, 1, 0), (2, K), "bf16", 3.0)
    w = draw((1110, 1, 2, 0), (K,), "f32")
    got, h = run_q8_1(dg, dev, x, res, w, K, K, h_is=h_is)
    href, y32, _ = reference(x, res, w)
    assert np.array_equal(got, orc.quantize_q8_1(y32).reshape(-1))
    if h_is != "none":
        assert torch.equal(h.float(), href.float())


@pytest.mark.parametrize("K", [1, 7, 8, 9, 63, 500, 2501, 8191, 20003, 40001])
@pytest.mark.parametrize("dtype,ydtype", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f32", "f16"),
                                          ("bf16", "f16"), ("f16", "bf16")])
def test_float_rows(dg, dev, K, dtype, ydtype):
    import torch
    M, ld, ldy = 4, K + 5, K + 3
    x = draw((1120, 1, K % 89, 0), (M, ld), dtype, 1.3)
    res = draw((1121, 1, K % 89, 0), (M, ld), dtype, 0.7)
    w = draw((1122, 1, K % 89, 0), (K,), "f32")
    h = torch.full((M, ld), 7.0, dtype=tdtype(dtype), device=dev)
    y = torch.full((M, ldy), 9.0, dtype=tdtype(ydtype), device=dev)
    dg.dg_rmsnorm(x.to(dev), w.to(dev), y, res=res.to(dev), h=h, eps=EPS, K=K)
    torch.cuda.synchronize()
    href, y32, y64 = reference(x[:, :K], res[:, :K], w)
    want = torch.from_numpy(y32).to(tdtype(ydtype))
    assert torch.equal(y.cpu()[:, :K].float(), want.float())
    assert (y.cpu()[:, K:].float() == 9.0).all() and (h.cpu()[:, K:].float() == 7.0).all()
    # against 64 bits: r, two products, the output's rounding, each half a step (first order, with a
    # quarter more for their products)
    rel = 1.25 * (3 * HALF_STEP["f32"] + (HALF_STEP[ydtype] if ydtype != "f32" else 0.0))
    err = np.abs(y.cpu()[:, :K].double().numpy() - y64)
    assert (err <= rel * np.abs(y64) + TINY[ydtype]).all()


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_misaligned_rows(dg, dev, orc, shift):
    """Operands aligned to their elements only."""
    import torch
    M, K = 3, 1024
    x, res = draw((1130, 1, 0, 0), (M, K), "f16"), draw((1130, 1, 1, 0), (M, K), "f16")
    w = draw((1130, 1, 2, 0), (K,), "f32")

    def off(t):
        b = torch.zeros(t.numel() + 16, dtype=t.dtype, device=dev)
        b[shift:shift + t.numel()] = t.to(dev).reshape(-1)
        return b[shift:shift + t.numel()].view(t.shape)
    hd = off(torch.zeros(M, K, dtype=torch.float16))
    Xq = torch.zeros(M * K // 32 * 36 + 16, dtype=torch.uint8, device=dev)[4 * shift:][:M * K // 32 * 36]
    dg.dg_rmsnorm_q8_1(off(x), off(w), Xq, res=off(res), h=hd, eps=EPS, K=K, M=M)
    torch.cuda.synchronize()
    href, y32, _ = reference(x, res, w)
    assert np.array_equal(Xq.cpu().numpy(), orc.quantize_q8_1(y32).reshape(-1))
    assert torch.equal(hd.cpu().float(), href.float())


def test_special_rows(dg, dev):
    """Zero rows give zeros; squares past binary32 do not overflow; infinities and NaN follow the formula and
    stay in their rows."""
    import torch
    K = 96
    x = torch.ones(6, K)
    x[0] = 0.0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    w = torch.full((K,), 2.0)
    y = torch.zeros(6, K, device=dev)
    dg.dg_rmsnorm(x.to(dev), w.to(dev), y, eps=EPS)
    Xq = torch.full((K // 32 * 36,), 0xA5, dtype=torch.uint8, device=dev)
    dg.dg_rmsnorm_q8_1(x[:1].to(dev), w.to(dev), Xq, eps=EPS)
    torch.cuda.synchronize()
    y = y.cpu()
    assert (y[0] == 0).all() and not Xq.cpu().any()
    _, y32, _ = reference(x, None, w)
    assert np.array_equal(y.numpy(), y32, equal_nan=True)
    assert torch.isnan(y[3, 5]) and (y[3, :5] == 0).all() and torch.isnan(y[4]).all()
    assert (y[5] == y[5, 0]).all() and abs(float(y[5, 0]) - 2.0) < 1e-4


@pytest.mark.parametrize("dtype,ydtype", [("f16", "f16"), ("f32", "f16"), ("bf16", "f16"), ("f16", "bf16")])
def test_each_rounding_of_many_values(dg, dev, dtype, ydtype):
    """About one value in 10^5 tells the binary32 product rounded to binary16 from the exact one rounded once, and so
    for the sum x + res: two million values have some of both."""
    import torch
    M, K = 700, 2821
    g = torch.Generator(device=dev).manual_seed(11)
    x = (torch.randn(M, K, device=dev, generator=g) * 3).to(tdtype(dtype))
    res = (torch.randn(M, K, device=dev, generator=g) * 0.01).to(tdtype(dtype))
    w = 1 + 0.2 * torch.randn(K, device=dev, generator=g)
    h = torch.zeros_like(x)
    y = torch.zeros(M, K, dtype=tdtype(ydtype), device=dev)
    dg.dg_rmsnorm(x, w, y, res=res, h=h, eps=EPS)
    torch.cuda.synchronize()
    href, y32, _ = reference(x.cpu(), res.cpu(), w.cpu())
    assert torch.equal(h.cpu().float(), href.float())
    assert torch.equal(y.cpu().float(), torch.from_numpy(y32).to(tdtype(ydtype)).float())


@pytest.mark.parametrize("M,K", [(70000, 64), ((1 << 21) + 3, 8)])   # the second in two launches
def test_many_rows(dg, dev, M, K):
    import torch
    x = torch.randn(M, K, device=dev, generator=torch.Generator(device=dev).manual_seed(5))
    w = torch.ones(K, device=dev)
    y = torch.zeros(M, K, device=dev)
    dg.dg_rmsnorm(x, w, y, eps=EPS)
    torch.cuda.synchronize()
    _, y32, _ = reference(x.cpu(), None, w.cpu())
    assert np.array_equal(y.cpu().numpy(), y32)


def test_many_rows_in_place_into_q8_1(dg, dev, orc):
    import torch
    M, K = (1 << 21) + 3, 32
    g = torch.Generator(device=dev).manual_seed(6)
    x = torch.randn(M, K, device=dev, generator=g).bfloat16()
    res = torch.randn(M, K, device=dev, generator=g).bfloat16()
    h0 = (x.float() + res.float()).bfloat16()
    w = torch.ones(K, device=dev)
    Xq = torch.zeros(M * 36, dtype=torch.uint8, device=dev)
    dg.dg_rmsnorm_q8_1(x, w, Xq, res=res, h=res, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(res, h0)
    for at in (0, (1 << 21) - 2):   # the first rows, and those across the launches' border
        _, y32, _ = reference(h0[at:at + 5].cpu(), None, w.cpu())
        assert np.array_equal(Xq.view(M, 36)[at:at + 5].cpu().numpy(), orc.quantize_q8_1(y32))


def test_empty(dg, dev):
    import torch
    x, w = torch.zeros(4, 64, device=dev), torch.ones(64, device=dev)
    y = torch.full((4, 64), 3.0, device=dev)
    dg.dg_rmsnorm(x, w, y, M=0)
    dg.dg_rmsnorm(x, w, y, K=0)
    torch.cuda.synchronize()
    assert (y == 3.0).all()


def test_operands_of_other_shapes_are_refused(dg, dev):
    import torch
    x = torch.ones(4, 64, device=dev)
    y = torch.empty_like(x)
    wide = torch.ones(4, 72, device=dev)
    with pytest.raises(ValueError, match="rows of 72"):
        dg.dg_rmsnorm(x, x[0], y, res=wide)
    with pytest.raises(ValueError, match="rows of 72"):
        dg.dg_rmsnorm(x, x[0], y, res=x, h=wide)
    with pytest.raises(ValueError, match="3 dimensions"):
        dg.dg_rmsnorm(x.view(2, 2, 64), x[0], y)
    with pytest.raises(ValueError, match="3 dimensions"):
        dg.dg_sample_rows(x.view(2, 2, 64), x[:, 0].contiguous(), torch.zeros(4, dtype=torch.int64, device=dev))
    dg.dg_rmsnorm(wide, x[0], y, res=wide, K=64)   # rows of 72, 64 used
    r = np.float32(1.0 / np.sqrt(4.0 + np.float64(np.float32(EPS))))   # h = 2 in every place
    assert torch.equal(y.cpu(), torch.full((4, 64), float(np.float32(2.0) * r)))
