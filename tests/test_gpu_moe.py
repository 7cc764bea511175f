"""The router and the routed experts against their definitions in 64 bits (GPU).

Router: scores, ranks and sums are binary64 on both sides, so the choice is
compared exactly and a weight is off by one rounding to binary32 (and the few
binary64 roundings below it).

Experts: the hidden columns that the call leaves in its workspace are compared
with the gated product in 64 bits under test_gpu_glu's tolerance t of that
product: a code may differ only where the exact quotient h/d lies within
(t + |h/d| t_max/127)/d of a rounding border, t_max the tolerance of the block's
largest value.  The output is then compared with the weighted sum of the down
products of the hidden columns as stored: a product of N/32 block terms passes
at most N/32 + 16 additions, the weighted sum k more roundings of products and
k of sums, then one rounding to the output type.
"""
import math

import numpy as np
import pytest

import synth
from tests.test_gpu_glu import ACTS, act64, columns, dev_u8, sums

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
HALF = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half the smallest subnormal
TYPES = ("f32", "f16", "bf16")


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


# ---- the router -------------------------------------------------------------------------------

def route64(x, k, score, bias, renorm, scale):
    M, E = x.shape
    ids, w = np.full((M, k), -1, np.int32), np.zeros((M, k))
    for m in range(M):
        v = x[m].astype(np.float64)
        ok = v > -np.inf
        if score == "softmax":
            top = np.max(v[ok]) if ok.any() else 0.0
            with np.errstate(invalid="ignore"):
                s = np.where(ok, np.where(v == top, 1.0, np.exp(np.where(ok, v, 0.0) - top)), 0.0)
            s = s / (s.sum() if s.sum() > 0 else 1.0)
            rank = v
        else:
            with np.errstate(over="ignore"):
                s = 1 / (1 + np.exp(-v))
            rank = s
        if bias is not None:
            rank = s + bias.astype(np.float64)
        cand = [e for e in range(E) if ok[e] and rank[e] > -np.inf]
        cand = sorted(cand, key=lambda e: (-rank[e], e))[:k]
        t = s[cand]
        if renorm:
            t = t / t.sum() if t.sum() > 0 else np.zeros_like(t)
        ids[m, :len(cand)], w[m, :len(cand)] = cand, t * float(np.float32(scale))
    return ids, w


def run_route(dg, dev, x, k, **kw):
    import torch
    M = x.shape[0]
    guard = 64
    ib = torch.full((M * k + 2 * guard,), -9, dtype=torch.int32, device=dev)
    wb = torch.full((M * k + 2 * guard,), -9.0, device=dev)
    ids, w = ib[guard:guard + M * k].view(M, k), wb[guard:guard + M * k].view(M, k)
    if kw.get("bias") is not None:
        kw["bias"] = torch.from_numpy(kw["bias"]).to(dev)
    dg.dg_moe_route(x.to(dev), ids, w, **kw)
    torch.cuda.synchronize()
    for b in (ib, wb):
        assert (b[:guard] == -9).all() and (b[-guard:] == -9).all(), "wrote outside the rows"
    return ids.cpu().numpy(), w.cpu().numpy()


def check_route(dg, dev, x, k, E=None, **kw):
    E = E or x.shape[1]
    ids, w = run_route(dg, dev, x, k, E=E, **kw)
    want, w64 = route64(x[:, :E].float().numpy(), k, kw.get("score", "softmax"), kw.get("bias"), kw.get("renorm", True),
                        kw.get("scale", 1.0))
    assert np.array_equal(ids, want), f"row {np.nonzero((ids != want).any(1))[0][0]}"
    tol = STEP * (1 + 2.0 ** -20) * np.abs(w64) + 2.0 ** -149
    assert (np.abs(w - w64) <= tol).all()
    return ids, w


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (5, 64, 6), (70, 65, 8), (33, 128, 8), (9, 160, 64), (301, 256, 8),
                                   (6, 511, 10), (4, 1024, 32), (1030, 16, 4)])
def test_route(dg, dev, M, E, k, score, dtype):
    import torch
    g = np.random.default_rng((M, E, k))
    ld = E + (3 if M % 2 else 0)
    x = torch.from_numpy((g.standard_normal((M, ld)) * 2).astype(np.float32)).to(tdtype(dtype))   # 16-bit rows hold ties
    check_route(dg, dev, x, k, E=E, score=score, ld=ld)
    check_route(dg, dev, x, k, E=E, score=score, ld=ld, renorm=False, scale=2.5)
    bias = (g.standard_normal(E) * 0.3).astype(np.float32)
    check_route(dg, dev, x, k, E=E, score=score, ld=ld, bias=bias, scale=-0.5)


def test_route_ties_go_to_the_lowest(dg, dev):
    import torch
    for E in (7, 64, 130, 1000):
        ids, _ = check_route(dg, dev, torch.zeros(3, E), min(E, 9))
        assert (ids == np.arange(min(E, 9))).all()
        x = torch.zeros(2, E)
        x[0, E // 2], x[1, ::2] = -0.0, -0.0
        check_route(dg, dev, x, 3)
        check_route(dg, dev, x, 3, score="sigmoid", bias=np.zeros(E, np.float32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_special_values(dg, dev, score):
    """Masked experts, rows with fewer experts than k or none, NaN, infinities, scores that vanish, a bias of -infinity."""
    import torch
    inf, nan = float("inf"), float("nan")
    E, k = 70, 4
    rows = [[-inf] * E, [nan] * E, [-inf] * 69 + [3.0], [1.0, nan, 2.0] + [-inf] * 67, [inf] + [0.0] * 69,
            [inf, 1.0, inf, -inf] + [0.5] * 66, [inf] * E, [-1e4] * E, [-1e30] * 3 + [-inf] * 67, [3e38] * 2 + [-3e38] * 68,
            [nan if e % 2 else float(e) for e in range(E)]]
    x = torch.tensor(rows)
    for renorm in (True, False):
        check_route(dg, dev, x, k, score=score, renorm=renorm)
        bias = np.linspace(-1, 1, E).astype(np.float32)
        bias[[5, 69]], bias[6] = -np.inf, np.nan
        check_route(dg, dev, x, k, score=score, renorm=renorm, bias=bias)
    check_route(dg, dev, x.bfloat16(), k, score=score)


# ---- the experts ------------------------------------------------------------------------------

class Layer:
    """Experts in both layouts, columns, and the definition's sums."""

    def __init__(self, dg, dev, orc, fmt, key, E, N, K, M, ids, act="silu"):
        import torch
        self.dg, self.dev, self.fmt, self.E, self.N, self.K, self.M, self.act = dg, dev, fmt, E, N, K, M, act
        self.ids = np.asarray(ids, np.int32).reshape(M, -1)
        self.k = self.ids.shape[1]
        quant = orc.quantize_q4_0 if fmt == "q4_0" else orc.quantize_q8_0
        self.rows, self.tiles = {}, {}
        for i, (n, r, c, s) in enumerate((("Wg", N, K, 2.0), ("Wu", N, K, 1.0), ("Wd", K, N, 1.0))):
            w = quant(synth.normal_f32((key, 0, i, 0), (E * r, c), s / math.sqrt(c)))
            self.rows[n] = np.ascontiguousarray(w).reshape(E, -1)
            t = torch.empty(getattr(dg, f"dg_{fmt}_tiles_bytes")(E * r, c), dtype=torch.uint8, device=dev)
            self.tiles[n] = getattr(dg, f"dg_repack_{fmt}_tiles")(dev_u8(dev, w), t, E * r, c)
        self.Xq = np.ascontiguousarray(orc.quantize_q8_1(synth.normal_f32((key, 1, 0, 0), (M, K), 1.5))).reshape(M, -1)
        g = np.random.default_rng(key)
        self.w = g.random((M, self.k)).astype(np.float32) - np.float32(0.2)

    def run(self, out="f32", rows=None, fill=0xA5):
        """(Y, hidden columns [M][k][N/32*36]) of tokens `rows`."""
        import torch
        rows = np.arange(self.M) if rows is None else np.asarray(rows)
        M, dev = len(rows), self.dev
        guard = 256
        buf = torch.full((M * self.K + 2 * guard,), 3.0, dtype=tdtype(out), device=dev)
        Y = buf[guard:guard + M * self.K].view(M, self.K)
        need = self.dg.dg_moe_workspace_bytes(self.N, self.K, M, self.k)
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=dev)
        t = [torch.from_numpy(np.ascontiguousarray(v[rows])).to(dev) for v in (self.Xq, self.ids, self.w)]
        getattr(self.dg, f"dg_moe_{self.fmt}")(self.tiles["Wg"], self.tiles["Wu"], self.tiles["Wd"], t[0], t[1], t[2], Y, self.N,
                                               self.K, M, self.E, act=self.act, ws=ws[:need])
        torch.cuda.synchronize()
        assert (buf[:guard] == 3).all() and (buf[-guard:] == 3).all(), "wrote outside Y"
        assert (ws[need:] == fill).all(), "wrote behind the workspace"
        H = ws[:M * self.k * (self.N // 32) * 36].cpu().numpy().reshape(M, self.k, -1)
        return Y.float().cpu().numpy(), H

    def slots(self):
        return [(m, j, int(e)) for m, r in enumerate(self.ids) for j, e in enumerate(r) if 0 <= e < self.E]

    def check_hidden(self, H):
        N, K, nb = self.N, self.K, self.N // 32
        for e in sorted({e for _, _, e in self.slots()}):
            mine = [(m, j) for m, j, f in self.slots() if f == e]
            X = self.Xq[[m for m, _ in mine]]
            (g, ga), (u, ua) = (sums(self.fmt, self.rows[n][e], X, N, K, len(mine)) for n in ("Wg", "Wu"))
            n = (K // 32 + 16) * STEP
            with np.errstate(over="ignore"):
                a, z = act64(self.act, g)
            dg, du = n * ga, n * ua
            tol = 1.2 * dg * (np.abs(u) + du) + np.abs(a) * du + (9 + 4 * z) * STEP * np.abs(a * u) * 1.01 + 2.0 ** -126
            h, tol = (a * u).reshape(len(mine), nb, 32), tol.reshape(len(mine), nb, 32)
            top = np.abs(h).argmax(-1)[..., None]
            amax, tmax = np.take_along_axis(np.abs(h), top, -1), tol.max(-1, keepdims=True)
            d, dt = amax / 127, tmax / 127 + STEP * amax / 127
            stored = np.stack([H[m, j] for m, j in mine])
            d16, q = columns(stored, len(mine), N)
            assert (np.abs(d16[..., None] - d) <= dt + 2.0 ** -11 * (d + dt) + 2.0 ** -25).all(), "scales"
            t = np.divide(h, d, out=np.zeros_like(h), where=d > 0)
            near = np.where(d > 0, (tol + np.abs(t) * dt) / np.where(d > 0, d, 1) * 1.01 + 2 * STEP * np.abs(t), 0)
            lo, hi = (np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127) for v in (t - near, t + near))
            assert ((q >= lo) & (q <= hi)).all(), "codes"
            assert (lo == hi).mean() > 0.9, "the tolerance decides nothing"
            s16 = stored.reshape(len(mine), nb, 36)[..., 2:4].copy().view(np.float16).astype(np.float64)[..., 0]
            s64 = d16 * q.sum(-1)      # from the stored d, whose rounding the stored s does not share
            assert (np.abs(s16 - s64) <= 2.0 ** -10 * np.abs(s64) * 1.01 + 2.0 ** -24 * (1 + np.abs(q.sum(-1)))).all(), "sums"

    def check_output(self, Y, H, out="f32"):
        y, tol = np.zeros((self.M, self.K)), np.zeros((self.M, self.K))
        mag = np.zeros((self.M, self.K))
        for e in sorted({e for _, _, e in self.slots()}):
            mine = [(m, j) for m, j, f in self.slots() if f == e]
            p, pa = sums(self.fmt, self.rows["Wd"][e], np.stack([H[m, j] for m, j in mine]), self.K, self.N, len(mine))
            for i, (m, j) in enumerate(mine):
                w = float(self.w[m, j])
                y[m] += w * p[i]
                tol[m] += abs(w) * (self.N // 32 + 16) * STEP * pa[i]
                mag[m] += abs(w) * pa[i]
        tol = tol + (self.k + 1) * STEP * mag * 1.01 + HALF[out] * (np.abs(y) + tol) * 1.01 + TINY[out] + 2.0 ** -140
        err = np.abs(Y - y)
        assert (err <= tol).all(), f"worst {np.max(err / tol):.2f} of the tolerance"

    def check(self, out="f32"):
        Y, H = self.run(out)
        self.check_hidden(H)
        self.check_output(Y, H, out)
        return Y, H


def distinct(key, E, M, k):
    g = np.random.default_rng(key)
    return np.stack([g.permutation(E)[:k] for _ in range(M)])


# (E, N, K, M, k): workgroups by slot and by expert; one column to several tiles of columns of one expert; rows of one
# group of 256 columns; columns that fill LDS in one pass and in several; enough workgroups for several row groups each
SHAPES = [(1, 256, 256, 1, 1), (8, 512, 256, 1, 3), (4, 256, 512, 3, 2), (16, 256, 768, 20, 4), (2, 768, 1280, 40, 2),
          (64, 256, 256, 5, 4), (2, 256, 4352, 24, 1), (2, 4608, 256, 20, 1), (3, 512, 512, 7, 3), (32, 256, 512, 33, 1),
          (64, 1280, 256, 60, 4), (64, 256, 2560, 60, 4), (16, 256, 256, 200, 4)]


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("E,N,K,M,k", SHAPES)
def test_definition(dg, dev, orc, fmt, E, N, K, M, k):
    c = Layer(dg, dev, orc, fmt, 1300 + E + M, E, N, K, M, distinct(M, E, M, k), act=ACTS[(E + M) % 4])
    Y, H = c.check()
    again, H2 = c.run(fill=0)
    assert np.array_equal(Y, again)
    for m, j, _ in c.slots():
        assert np.array_equal(H[m, j], H2[m, j])


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("act", ACTS)
def test_activations_and_types(dg, dev, orc, fmt, act):
    c = Layer(dg, dev, orc, fmt, 1400, 4, 512, 512, 5, distinct(1, 4, 5, 2), act=act)
    Y, H = c.check()
    for out in ("f16", "bf16"):
        Y16, H16 = c.run(out)
        import torch
        assert np.array_equal(Y16, torch.from_numpy(Y).to(tdtype(out)).float().numpy()), "not one rounding of the sums"


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_rows_without_experts_and_odd_ids(dg, dev, orc, fmt):
    """Slots and tokens without an expert, ids outside the range, the same expert twice in a token; every expert unused but
    one; nothing routed at all."""
    E, M = 6, 9
    ids = distinct(5, E, M, 3)
    ids[0], ids[4, 1], ids[5] = -1, E, [-(1 << 31), (1 << 31) - 1, 2]
    ids[6], ids[7], ids[8] = [3, 3, 3], [1, 3, 1], [-1, 0, -1]
    c = Layer(dg, dev, orc, fmt, 1500, E, 512, 256, M, ids)
    Y, H = c.check()
    assert not Y[0].any()
    c.w[(ids < 0) | (ids >= E)] = np.nan      # what slots without an expert hold, in the workspace too, does not count
    assert np.array_equal(Y, c.run(fill=0xFF)[0])
    one = Layer(dg, dev, orc, fmt, 1500, E, 512, 256, M, np.full((M, 3), 5))   # 27 columns of one expert
    one.check()
    many = Layer(dg, dev, orc, fmt, 1500, E, 512, 256, 60, np.where(np.arange(180).reshape(60, 3) % 7, ids[np.arange(60) % M], -1))
    Y, H = many.check()                        # past what one kernel makes of a token
    many.w[(many.ids < 0) | (many.ids >= E)] = np.inf
    assert np.array_equal(Y, many.run(fill=0xFF)[0])
    none = Layer(dg, dev, orc, fmt, 1500, E, 512, 256, M, np.full((M, 3), -1))
    Y, H = none.run()
    assert not Y.any() and (H == 0xA5).all()


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("k", [4, 20])
def test_an_expert_many_times_in_few_tokens(dg, dev, orc, fmt, k):
    """More columns of one expert than tokens: all slots the same, and two experts in turn; few slots a token and many."""
    for ids in (np.full((4, k), 2), np.arange(4 * k).reshape(4, k) % 2 * 3):
        for E in (6, 200):     # workgroups by expert and by slot
            Layer(dg, dev, orc, fmt, 1800, E, 256, 512, 4, ids).check()


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_a_token_does_not_depend_on_the_others(dg, dev, orc, fmt):
    """Alone, in a batch and beside others of its expert in any number: the same bits (columns in one pass and several)."""
    for E, N, K, M, k in ((3, 512, 4608, 45, 1), (3, 4608, 512, 30, 2), (8, 256, 512, 12, 3)):
        c = Layer(dg, dev, orc, fmt, 1600, E, N, K, M, distinct(3, E, M, k))
        Y, H = c.run()
        for rows in ([0], [M - 1], [M // 2, 1], list(range(3, M - 1)), list(range(M))[::-1]):
            Y1, H1 = c.run(rows=rows)
            assert np.array_equal(Y1, Y[rows]) and np.array_equal(H1, H[rows])


def test_most_slots(dg, dev, orc):
    """As many slots as a call takes, over few and over many experts."""
    for E, M, k in ((2, 2048, 2), (1024, 64, 64)):
        c = Layer(dg, dev, orc, "q4_0", 1700, E, 256, 256, M, distinct(9, E, M, k))
        c.check()


def test_experts_past_32_bit_offsets(dg, dev):
    """The last of experts whose matrices span more than 2^33 bytes gives what the same weights in the first place give."""
    import torch
    E, N, K = 140, 14336, 4096
    g = torch.Generator(device=dev).manual_seed(4)

    def stack(rows, cols):
        w = torch.empty(rows * (cols // 32) * 34, dtype=torch.uint8, device=dev)
        dg.dg_quantize_q8_0(torch.randn(rows, cols, device=dev, generator=g) / math.sqrt(cols), w, rows, cols)
        one = torch.empty(dg.dg_q8_0_tiles_bytes(rows, cols), dtype=torch.uint8, device=dev)
        dg.dg_repack_q8_0_tiles(w, one, rows, cols)
        all_ = torch.zeros(E * one.numel(), dtype=torch.uint8, device=dev)
        all_[:one.numel()], all_[-one.numel():] = one, one
        return all_
    Wg, Wd = stack(N, K), stack(K, N)
    assert Wg.numel() > 1 << 33
    for M in (1, 20):      # a token's down products with their sum, and by themselves
        Xq = torch.empty(M * K // 32 * 36, dtype=torch.uint8, device=dev)
        dg.dg_quantize_q8_1(torch.randn(M, K, device=dev, generator=g), Xq, M, K)
        w = torch.ones(M, 1, device=dev)
        ws = torch.zeros(dg.dg_moe_workspace_bytes(N, K, M, 1), dtype=torch.uint8, device=dev)
        Y = [torch.zeros(M, K, device=dev) for _ in range(3)]
        for y, e in zip(Y, (0, E - 1, E // 2)):
            ids = torch.full((M, 1), e, dtype=torch.int32, device=dev)
            dg.dg_moe_q8_0(Wg, Wg, Wd, Xq, ids, w, y, N, K, M, E, ws=ws)
        torch.cuda.synchronize()
        assert Y[0].abs().max() > 0.1 and torch.equal(Y[0], Y[1]) and not Y[2].any()


def test_empty_sizes(dg, dev):
    import torch
    u8 = torch.zeros(16, dtype=torch.uint8, device=dev)
    Y = torch.full((3, 256), 5.0, device=dev)
    ids, w = torch.zeros(3, 1, dtype=torch.int32, device=dev), torch.ones(3, 1, device=dev)
    dg.dg_moe_q4_0(u8, u8, u8, u8, ids, w, Y, N=0, K=256, M=3, E=2)
    torch.cuda.synchronize()
    assert not Y.any()
    Y.fill_(5.0)
    dg.dg_moe_q8_0(u8, u8, u8, u8, ids, w, Y, N=256, K=256, M=3, E=2, k=0)
    torch.cuda.synchronize()
    assert not Y.any()
    dg.dg_moe_q8_0(u8, u8, u8, u8, ids, w, Y, N=256, K=0, M=3, E=2)
    dg.dg_moe_q8_0(u8, u8, u8, u8, ids, w, Y, N=256, K=256, M=0, E=2)


def test_binding_refuses(dg, dev):
    import torch
    x, ids, w = torch.zeros(4, 8, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev), torch.zeros(4, 2, device=dev)
    with pytest.raises(ValueError, match="score"):
        dg.dg_moe_route(x, ids, w, score="relu")
    with pytest.raises(ValueError, match="weights holds"):
        dg.dg_moe_route(x, ids, w[:3])
    with pytest.raises(TypeError, match="ids has dtype"):
        dg.dg_moe_route(x, ids.long(), w)
    with pytest.raises(dg.DGError, match="DG_ERR_SHAPE"):
        dg.dg_moe_route(x, torch.zeros(4, 9, dtype=torch.int32, device=dev), torch.zeros(4, 9, device=dev))
    E, N, K, M = 2, 256, 256, 4
    W = torch.zeros(E * N * (K // 32) * 18, dtype=torch.uint8, device=dev)
    Xq, Y = torch.zeros(M * K // 32 * 36, dtype=torch.uint8, device=dev), torch.zeros(M, K, device=dev)
    ws = torch.zeros(dg.dg_moe_workspace_bytes(N, K, M, 2), dtype=torch.uint8, device=dev)
    call = lambda **kw: dg.dg_moe_q4_0(**(dict(Wg=W, Wu=W, Wd=W, Xq=Xq, ids=ids, weights=w, Y=Y, N=N, K=K, M=M, E=E, ws=ws) | kw))  # noqa: E731
    call()
    for kw, match in ((dict(Wd=W[16:]), "Wd holds"), (dict(Xq=Xq[:-4]), "Xq holds"), (dict(Y=Y[:3]), "Y holds"),
                      (dict(act="tanh"), "act must"), (dict(ids=ids.cpu()), "host tensor"), (dict(weights=w.half()), "weights has")):
        with pytest.raises((TypeError, ValueError), match=match):
            call(**kw)
    for kw, match in ((dict(ws=None), "WORKSPACE"), (dict(ws=ws[16:]), "WORKSPACE"), (dict(N=128, K=128), "SHAPE")):
        with pytest.raises(dg.DGError, match=match):
            call(**kw)
