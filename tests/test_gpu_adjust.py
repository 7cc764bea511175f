"""Penalties, biases and grammar masks on rows of logits (GPU).

Every operation of the definition is one binary32 operation on exactly known values, so the result is compared bit for
bit with a numpy statement of it, rounded once to the type.
"""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

F = np.float32
TYPES = ("f32", "f16", "bf16")


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def reference(x, C, a):
    """float32 rows of the definition; a: numpy arrays by name."""
    out = x[:, :C].astype(F).copy()
    for r in range(out.shape[0]):
        v = out[r]
        T = a["tokens"].shape[1] if a.get("tokens") is not None else 0
        n = int(np.clip(a["lens"][r], 0, T)) if a.get("lens") is not None else T
        p = int(np.clip(a["prompt_lens"][r], 0, n)) if a.get("prompt_lens") is not None else 0
        hist = a["tokens"][r] if T else np.zeros(0, np.int64)
        inside = lambda t: t[(t >= 0) & (t < C)]  # noqa: E731
        seen = np.unique(inside(hist[:n]))
        said, times = np.unique(inside(hist[p:n]), return_counts=True)
        rep = F(a["repetition"][r]) if a.get("repetition") is not None else F(1)
        with np.errstate(all="ignore"):
            if rep > 0:
                v[seen] = np.where(v[seen] > 0, v[seen] / rep, v[seen] * rep)
            f = F(a["frequency"][r]) if a.get("frequency") is not None else F(0)
            q = F(a["presence"][r]) if a.get("presence") is not None else F(0)
            v[said] = (v[said] - f * times.astype(F)) - q
            if a.get("bias") is not None:
                B = a["bias"].shape[1]
                last = {int(t): F(b) for t, b in list(zip(a["bias_ids"][r], a["bias"][r]))[
                    : int(np.clip(a["bias_lens"][r], 0, B)) if a.get("bias_lens") is not None else B] if 0 <= t < C}
                for t, b in last.items():
                    v[t] = v[t] + b
        if a.get("mask") is not None:
            bits = np.unpackbits(np.ascontiguousarray(a["mask"][r]).view(np.uint8), bitorder="little")[:C]
            v[bits == 0] = -np.inf
        assert v.dtype == F
    return out


def same(got, want, dtype):
    """Equal bits of two CPU tensors of the type, any NaN equal to any."""
    import torch
    bits = torch.int32 if dtype == "f32" else torch.int16
    eq = (got.view(bits) == want.view(bits)) | (got.isnan() & want.isnan())
    assert eq.all(), f"{int((~eq).sum())} differ, first at {torch.nonzero(~eq)[0].tolist()}"


def run(dg, dev, x, C, a, in_place=False, ldy=None, **kw):
    """x: CPU tensor [R][ld]; what the call makes of it, and checks of what it may not touch."""
    import torch
    R, ld = x.shape
    t = {n: torch.from_numpy(np.ascontiguousarray(v)).to(dev) for n, v in a.items() if v is not None}
    xd = x.to(dev)
    ldy = ld if in_place else ldy or C
    guard = 64
    buf = torch.full((R * ldy + 2 * guard,), 5.0, dtype=x.dtype, device=dev)
    y = xd if in_place else buf[guard:guard + R * ldy].view(R, ldy)
    dg.dg_adjust_rows(xd, y, C=C, ld=ld, ldy=ldy, **t, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert (buf[:guard] == 5).all() and (buf[-guard:] == 5).all() and (y[:, C:] == 5).all(), "wrote outside the rows"
        same(xd.cpu(), x, {torch.float32: "f32"}.get(x.dtype, "16"))
    else:
        same(y[:, C:].cpu().contiguous(), x[:, C:].contiguous(), {torch.float32: "f32"}.get(x.dtype, "16"))
    return y[:, :C].cpu().contiguous()


def draw(key, R, C, ld, T, B, dtype, mask=True):
    """Logits and adjustments of rows, histories with many repeats and tokens outside the vocabulary."""
    import torch
    g = np.random.default_rng(key)
    x = torch.from_numpy((g.standard_normal((R, ld)) * 4).astype(F)).to(tdtype(dtype))
    a = {}
    if T:
        tok = np.where(g.random((R, T)) < 0.5, g.integers(0, max(1, C // 50 + 1), (R, T)), g.integers(-3, C + 3, (R, T)))
        a["tokens"] = tok.astype(np.int32)
        a["lens"] = g.integers(-1, T + 3, R).astype(np.int32)
        a["prompt_lens"] = (a["lens"] // 2 + g.integers(-2, 3, R)).astype(np.int32)
        a["repetition"] = g.choice([1.0, 1.1, 1.37, 0.8], R).astype(F)
        a["frequency"] = (g.random(R) * 0.7 - 0.1).astype(F)
        a["presence"] = (g.random(R) * 0.7 - 0.1).astype(F)
    if B:
        a["bias_ids"] = g.integers(-2, C + 2, (R, B)).astype(np.int32)
        a["bias"] = (g.standard_normal((R, B)) * 5).astype(F)
        a["bias"][g.random((R, B)) < 0.2] = -np.inf
        a["bias_lens"] = g.integers(0, B + 2, R).astype(np.int32)
    if mask:
        a["mask"] = g.integers(-2 ** 31, 2 ** 31, (R, -(-C // 32) + 1)).astype(np.int32)
    return x, a


# chunk ends, words of the mask that end inside a chunk, odd strides (rows at every alignment), long histories
SHAPES = [(1, 1, 1, 0, 0), (3, 1, 5, 2, 1), (2, 31, 31, 40, 3), (5, 33, 37, 7, 70), (4, 1000, 1000, 513, 5),
          (3, 8191, 8195, 100, 9), (2, 8192, 8192, 3000, 300), (3, 8193, 8193, 64, 0), (7, 16391, 16392, 1, 33),
          (2, 32003, 32011, 20000, 40), (65, 4099, 4104, 65, 4), (1, 128256, 128256, 5000, 16), (2, 151937, 151937, 70, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C,ld,T,B", SHAPES)
def test_definition(dg, dev, R, C, ld, T, B, dtype):
    import torch
    for mask in (False, True):
        x, a = draw((R, C, T, B, mask), R, C, ld, T, B, dtype, mask)
        want = torch.from_numpy(reference(x.float().numpy(), C, a)).to(x.dtype)
        same(run(dg, dev, x, C, a, ldy=C + 3), want, dtype)
        same(run(dg, dev, x, C, a, in_place=True), want, dtype)


@pytest.mark.parametrize("off", [{"tokens", "lens", "prompt_lens"}, {"lens"}, {"prompt_lens"}, {"repetition"}, {"frequency"},
                                 {"presence"}, {"bias_ids", "bias", "bias_lens"}, {"bias_lens"}, {"mask"},
                                 {"repetition", "frequency", "presence"}, {"tokens", "lens", "prompt_lens", "bias_ids", "bias",
                                                                           "bias_lens", "mask"}])
def test_absent_arrays(dg, dev, off):
    import torch
    x, a = draw(77, 6, 9001, 9004, 300, 12, "f32")
    for n in off:
        a[n] = None
    same(run(dg, dev, x, 9001, a), torch.from_numpy(reference(x.numpy(), 9001, a)), "f32")


def test_nothing_to_do_copies(dg, dev):
    import torch
    for dtype in TYPES:
        x, _ = draw(3, 4, 10007, 10010, 0, 0, dtype)
        same(run(dg, dev, x, 10007, {}), x[:, :10007].contiguous(), dtype)
    st = dg.raw().dg_adjust_rows(1 << 20, 1 << 21, 0, 0, 5, 5, 5, None, None)   # no adjustments at all, no rows
    assert st == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(dg, dev, dtype):
    """Infinities, NaN, zeros and the type's extremes, in the history, with a bias, masked and not; penalties that are
    infinite, zero, negative or NaN."""
    import torch
    lim = torch.finfo(tdtype(dtype))
    special = [np.inf, -np.inf, np.nan, 0.0, -0.0, lim.max, lim.min, lim.tiny, -lim.tiny, lim.smallest_normal / 2, 1.0]
    C = 64
    reps = [1.0, 2.0, np.inf, 0.0, -1.5, np.nan, 1e-30]
    pens = [0.0, 0.5, np.inf, -np.inf, np.nan, -2.0, 1e38]
    x = torch.tensor(special + [1.5] * (C - len(special)), dtype=torch.float32).to(tdtype(dtype)).repeat(len(reps), 1)
    n = len(reps)
    tok = np.tile(np.concatenate([np.arange(C), np.arange(C // 2), np.arange(5)]).astype(np.int32), (n, 1))
    a = dict(tokens=tok, lens=None, prompt_lens=np.full(n, 20, np.int32), repetition=np.array(reps, F),
             frequency=np.array(pens, F), presence=np.array(pens[::-1], F))
    for bias in (None, np.inf, -np.inf, np.nan):
        if bias is not None:
            a["bias_ids"], a["bias"] = np.tile(np.arange(12, dtype=np.int32), (n, 1)), np.full((n, 12), bias, F)
        for mask in (None, 0x55555555, 0):
            a["mask"] = None if mask is None else np.full((n, 2), mask, np.int32)
            with np.errstate(all="ignore"):
                want = torch.from_numpy(reference(x.float().numpy(), C, a)).to(x.dtype)
            same(run(dg, dev, x, C, a), want, dtype)
            if mask == 0:
                assert torch.isneginf(want).all()


def test_last_bias_of_a_token_counts(dg, dev):
    import torch
    C, B = 20000, 5000
    g = np.random.default_rng(5)
    x = torch.from_numpy(g.standard_normal((3, C)).astype(F))
    a = dict(bias_ids=g.integers(0, 40, (3, B)).astype(np.int32) * 500, bias=g.standard_normal((3, B)).astype(F))
    want = torch.from_numpy(reference(x.numpy(), C, a))
    for _ in range(3):
        same(run(dg, dev, x, C, a), want, "f32")


def test_counts_are_exact(dg, dev):
    """One token a hundred thousand times, beside its neighbours."""
    import torch
    C, T = 9000, 100003
    tok = np.full((2, T), 8192, np.int32)
    tok[1, ::3] = 8191
    a = dict(tokens=tok, prompt_lens=np.array([3, 50001], np.int32), frequency=np.array([0.25, 0.125], F),
             presence=np.array([0.5, 0.25], F), repetition=np.array([1.5, 1.25], F))
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((2, C)).astype(F))
    same(run(dg, dev, x, C, a), torch.from_numpy(reference(x.numpy(), C, a)), "f32")


def test_rows_past_32_bit_offsets(dg, dev):
    """Rows whose elements lie beyond 2^32 bytes and 2^31 elements."""
    import torch
    ld, C, R = (1 << 30) + 64, 5000, 3
    x = torch.empty(2 * ld + C, dtype=torch.float16, device=dev)
    want = []
    g = np.random.default_rng(8)
    a = dict(tokens=g.integers(0, C, (R, 50)).astype(np.int32), repetition=np.full(R, 1.3, F), presence=np.full(R, 0.5, F))
    rows = torch.from_numpy(g.standard_normal((R, C)).astype(F)).half()
    for r in range(R):
        x[r * ld:r * ld + C] = rows[r].to(dev)
    y = torch.zeros(R, C, dtype=torch.float16, device=dev)
    t = {n: torch.from_numpy(v).to(dev) for n, v in a.items()}
    dg.dg_adjust_rows(x, y, R=R, C=C, ld=ld, **t)
    torch.cuda.synchronize()
    want = torch.from_numpy(reference(rows.float().numpy(), C, a)).half()
    same(y.cpu(), want, "f16")


def test_binding_refuses(dg, dev):
    import torch
    x = torch.zeros(4, 100, device=dev)
    i = torch.zeros(4, 10, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="y holds"):
        dg.dg_adjust_rows(x, torch.zeros(3, 100, device=dev))
    with pytest.raises(TypeError, match="y has dtype"):
        dg.dg_adjust_rows(x, x.half())
    with pytest.raises(TypeError, match="tokens has dtype"):
        dg.dg_adjust_rows(x, x, tokens=i.long())
    with pytest.raises(ValueError, match="tokens holds"):
        dg.dg_adjust_rows(x, x, tokens=i[:3])
    with pytest.raises(ValueError, match="host tensor"):
        dg.dg_adjust_rows(x, x, repetition=torch.ones(4))
    with pytest.raises(ValueError, match="contiguous"):
        dg.dg_adjust_rows(x, x, tokens=i.t())
    with pytest.raises(dg.DGError, match="DG_ERR_ARG"):
        dg.dg_adjust_rows(x, x, bias_ids=i)
    with pytest.raises(dg.DGError, match="DG_ERR_SHAPE"):
        dg.dg_adjust_rows(x, x, mask=torch.zeros(4, 3, dtype=torch.int32, device=dev))
