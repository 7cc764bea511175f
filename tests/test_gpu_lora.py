"""Low-rank adapters of many requests against their definition in 64 bits (GPU).

Tolerance, derived per output.  h[r] is a sum of K products of stored values:
a product is rounded by at most 2^-24 of itself (the products of two 16-bit
values are exact) and then passes at most K additions, each rounded by 2^-24
of a partial sum that is at most ha[r] = sum |A x|: |dh| <= (K + 1) 2^-24 ha.
The sum over r adds (R + 1) 2^-24 of sum |B| (|h| + |dh|) likewise, the scale
and the addition to the base one rounding each.
"""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
TYPES = ("f32", "f16", "bf16")


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


class Case:
    def __init__(self, key, M, N, K, R, L, x="f32", w="bf16", ld=None, ranks=None, scale=True, base=True, adapter=None):
        import torch
        g = np.random.default_rng(key)
        self.M, self.N, self.K, self.R, self.L, self.ld = M, N, K, R, L, ld or K
        normal = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32))  # noqa: E731
        self.x = normal(M, self.ld).to(tdtype(x))
        self.A = (normal(L, R, K) / max(K, 1) ** 0.5).to(tdtype(w))
        self.B = normal(L, N, R).to(tdtype(w))
        a = g.integers(-1, L + 1, M) if adapter is None else np.asarray(adapter)
        self.adapter = torch.from_numpy(a.astype(np.int32))
        self.scale = torch.from_numpy((g.random(L) * 2 - 0.5).astype(np.float32)) if scale else None
        self.ranks = torch.from_numpy(np.asarray(ranks, np.int32)) if ranks is not None else None
        self.base = normal(M, N) if base else None

    def definition(self):
        """(Y, the tolerance) in 64 bits."""
        y, tol = np.zeros((self.M, self.N)), np.zeros((self.M, self.N))
        for m, a in enumerate(self.adapter.tolist()):
            if 0 <= a < self.L:
                r = self.R if self.ranks is None else min(max(int(self.ranks[a]), 0), self.R)
                A, B = self.A[a, :r].double().numpy(), self.B[a, :, :r].double().numpy()
                x = self.x[m, :self.K].double().numpy()
                h, dh = A @ x, (self.K + 1) * STEP * (np.abs(A) @ np.abs(x))
                s = 1.0 if self.scale is None else float(self.scale[a])
                mag = np.abs(B) @ (np.abs(h) + dh)
                y[m] = s * (B @ h)
                tol[m] = abs(s) * (np.abs(B) @ dh + (r + 2) * STEP * mag)
        if self.base is not None:
            y += self.base.double().numpy()
        return y, tol * 1.01 + STEP * np.abs(y) * 1.01 + 2.0 ** -140

    def run(self, dg, dev, in_place=False, fill=None):
        import torch
        put = lambda t: None if t is None else t.to(dev)  # noqa: E731
        guard = 64
        buf = torch.full((self.M * self.N + 2 * guard,), -7.0, device=dev)
        Y = buf[guard:guard + self.M * self.N].view(self.M, self.N)
        base = put(self.base)
        if in_place:
            Y.copy_(base)
            base = Y
        need = dg.dg_lora_workspace_bytes(self.M, self.K, self.R)
        ws = torch.full((need,), 0xA5 if fill is None else fill, dtype=torch.uint8, device=dev)
        dg.dg_lora_rows(put(self.x), put(self.A), put(self.B), put(self.adapter), Y, base=base, scale=put(self.scale),
                        ranks=put(self.ranks), M=self.M, N=self.N, K=self.K, R=self.R, L=self.L, ld=self.ld, ws=ws)
        torch.cuda.synchronize()
        assert (buf[:guard] == -7).all() and (buf[-guard:] == -7).all(), "wrote outside Y"
        return Y.cpu().numpy()

    def check(self, dg, dev, **kw):
        got = self.run(dg, dev, **kw)
        want, tol = self.definition()
        err = np.abs(got - want)
        worst = np.unravel_index(np.argmax(err / tol), err.shape)
        assert (err <= tol).all(), f"at {worst}: got {got[worst]!r}, expected {want[worst]!r}, tolerance {tol[worst]:.3e}"
        return got


# one row to many, past what is grouped together (1024), every kind of rank, odd numbers of outputs, short and long rows
# of K
SHAPES = [(1, 1, 8, 8, 1), (1, 300, 4096, 16, 3), (2, 255, 520, 24, 2), (3, 1001, 8, 8, 2), (5, 257, 1032, 40, 1),
          (7, 64, 2048, 64, 4), (16, 513, 768, 16, 5), (17, 130, 4104, 128, 3), (33, 77, 264, 8, 40), (64, 100, 512, 32, 2),
          (65, 1030, 256, 16, 9), (130, 45, 1000, 72, 3), (200, 515, 136, 32, 7), (1, 97, 16392, 512, 2), (3, 31, 24, 504, 1),
          (1100, 70, 64, 8, 3), (2049, 33, 40, 16, 5), (4, 2101, 1032, 56, 3), (4, 2101, 1032, 32, 3), (2, 1500, 5000, 24, 2), (6, 1024, 8200, 8, 3), (128, 1024, 72, 8, 6), (129, 1024, 72, 8, 6)]


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("w", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,R,L", SHAPES)
def test_definition(dg, dev, M, N, K, R, L, x, w):
    Case((M, N, K, R), M, N, K, R, L, x, w).check(dg, dev)


@pytest.mark.parametrize("M,N,K,R,L", [(1, 300, 264, 16, 2), (40, 129, 520, 32, 4)])
def test_options(dg, dev, M, N, K, R, L):
    key = (M, 7)
    got = Case(key, M, N, K, R, L).check(dg, dev)
    assert np.array_equal(got, Case(key, M, N, K, R, L).check(dg, dev, in_place=True))
    Case(key, M, N, K, R, L, scale=False).check(dg, dev)
    Case(key, M, N, K, R, L, base=False).check(dg, dev)
    Case(key, M, N, K, R, L, ld=K + 16).check(dg, dev)
    c = Case(key, M, N, K, R, L, base=False, adapter=np.full(M, -1))
    assert not c.run(dg, dev).any()
    c = Case(key, M, N, K, R, L, adapter=np.where(np.arange(M) % 2, L, -(1 << 31)))
    assert np.array_equal(c.run(dg, dev), c.base.numpy())


@pytest.mark.parametrize("N,R", [(203, 40), (3001, 40), (45, 136), (203, 32), (3001, 32), (1200, 16)])
def test_ranks(dg, dev, N, R):
    """Every rank from none to all and beyond; what lies past a rank is not read as a number."""
    ranks = [0, 1, 2, 7, 8, 9, 15, 16, 23, 24, 25, 31, 32, 33, 40, 41, -3, 1 << 30]
    L = len(ranks)
    for x in TYPES:
        c = Case(11, 3 * L, N, 392, R, L, x, ranks=ranks, adapter=np.arange(3 * L) % L)
        want = c.check(dg, dev)
        for a, r in enumerate(ranks):
            r = min(max(r, 0), R)
            c.A[a, r:] = float("nan")
            c.B[a, :, r:] = float("inf")
        assert np.array_equal(want, c.run(dg, dev, fill=0xFF))   # a workspace of NaN


def test_no_columns_and_no_adapters(dg, dev):
    c = Case(3, 5, 70, 0, 16, 2, ld=8)
    assert np.array_equal(c.run(dg, dev), c.base.numpy())
    c = Case(3, 5, 70, 64, 16, 0, adapter=np.zeros(5))
    assert np.array_equal(c.run(dg, dev), c.base.numpy())


@pytest.mark.parametrize("N,K,R", [(333, 1544, 48), (2101, 1544, 16), (2101, 264, 64), (2101, 1544, 32)])
@pytest.mark.parametrize("pattern", ["one", "runs", "mixed", "distinct"])
def test_a_row_does_not_depend_on_the_others(dg, dev, pattern, N, K, R):
    """However the adapters of the batch are spread, each row is the row of a call of its own, bit for bit."""
    M, L = 71, 9
    adapter = {"one": np.full(M, 4), "runs": np.arange(M) // 8, "mixed": np.random.default_rng(2).integers(-1, L, M),
               "distinct": np.arange(M) % L}[pattern]
    c = Case(21, M, N, K, R, L, "bf16", adapter=adapter)
    got = c.check(dg, dev)
    assert np.array_equal(got, c.run(dg, dev))
    for m in (0, 1, 13, 70):
        one = Case(21, M, N, K, R, L, "bf16", adapter=adapter)
        one.M, one.x, one.adapter, one.base = 1, c.x[m:m + 1], c.adapter[m:m + 1], c.base[m:m + 1]
        assert np.array_equal(one.run(dg, dev)[0], got[m])


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("w", ["f16", "bf16"])
def test_subnormal_values(dg, dev, x, w):
    """Weights and rows below the smallest normal number of their type count for what they are."""
    import torch
    c = Case(31, 5, 100, 128, 16, 2, x, w, adapter=[0, 1, 0, 1, 1], base=False, scale=False)
    tiny = torch.finfo(tdtype(w)).smallest_normal
    c.A = (c.A.float().sign() * tiny * 0.375).to(tdtype(w))
    c.x = torch.full_like(c.x, 1.0)
    c.B = c.B.float().sign().to(tdtype(w)) * (2.0 ** 100 if w == "bf16" else 2.0 ** 10)
    c.check(dg, dev)
    assert np.abs(c.definition()[0]).max() > 100 * c.definition()[1].max()
    if x != "f32":
        c.A, c.x = c.A.float().sign().to(tdtype(w)), (c.x.float() * torch.finfo(tdtype(x)).smallest_normal / 4).to(tdtype(x))
        c.check(dg, dev)


def test_infinities_stay_in_their_row(dg, dev):
    c = Case(5, 40, 100, 256, 16, 3, adapter=np.arange(40) % 3)
    want = c.run(dg, dev)
    c.x[7, 3], c.x[20, 250] = float("inf"), float("nan")
    got = c.run(dg, dev)
    clean = [m for m in range(40) if m not in (7, 20)]
    assert np.array_equal(got[clean], want[clean]) and not np.isfinite(got[[7, 20]]).any()


def test_very_many_rows(dg, dev):
    """More rows than a launch takes, of the first product and of the windows: one adapter, rows without it among them."""
    M, N, K, R = 140000, 9, 16, 8
    c = Case(41, M, N, K, R, 1, "bf16", adapter=np.arange(M) % 5 % 2 - 1)
    got = c.run(dg, dev)
    x, A, B = c.x.double().numpy(), c.A[0].double().numpy(), c.B[0].double().numpy()
    has, s = (c.adapter.numpy() == 0)[:, None], abs(float(c.scale[0]))
    h, dh = x @ A.T, (K + 1) * STEP * (np.abs(x) @ np.abs(A).T)
    want = c.base.double().numpy() + np.where(has, float(c.scale[0]) * (h @ B.T), 0.0)
    tol = np.where(has, s * (dh @ np.abs(B).T + (R + 2) * STEP * ((np.abs(h) + dh) @ np.abs(B).T)), 0.0) + STEP * np.abs(want)
    assert (np.abs(got - want) <= 1.01 * tol).all()


def test_adapters_past_32_bit_offsets(dg, dev):
    """The last of adapters whose weights span more than 2^32 bytes, each."""
    import torch
    L, R, K, N, M = 3, 512, 2 << 20, 1 << 21, 2
    A = torch.zeros(L, R, K, dtype=torch.bfloat16, device=dev)
    B = torch.zeros(L, N, R, dtype=torch.bfloat16, device=dev)
    A[2, 500, K - 8:], B[2, N - 1, 500] = 1.0, 2.0
    x = torch.ones(M, K, dtype=torch.bfloat16, device=dev)
    Y = torch.zeros(M, N, device=dev)
    ad = torch.tensor([2, 0], dtype=torch.int32, device=dev)
    ws = torch.zeros(dg.dg_lora_workspace_bytes(M, K, R), dtype=torch.uint8, device=dev)
    dg.dg_lora_rows(x, A, B, ad, Y, ws=ws)
    torch.cuda.synchronize()
    assert float(Y[0, N - 1]) == 16.0 and float(Y.abs().sum()) == 16.0


def test_binding_refuses(dg, dev):
    import torch
    c = Case(1, 4, 50, 64, 16, 2)
    t = {n: getattr(c, n).to(dev) for n in ("x", "A", "B", "adapter", "base")}
    Y, ws = torch.zeros(4, 50, device=dev), torch.zeros(dg.dg_lora_workspace_bytes(4, 64, 16), dtype=torch.uint8, device=dev)
    call = lambda **kw: dg.dg_lora_rows(**(t | dict(Y=Y, ws=ws) | kw))  # noqa: E731
    call()
    for kw, match in ((dict(B=t["B"].half()), "B has dtype"), (dict(adapter=t["adapter"][:3]), "adapter holds"),
                      (dict(Y=Y[:3]), "Y holds|base holds"), (dict(scale=torch.ones(2)), "host tensor"), (dict(x=t["x"].t()), "x")):
        with pytest.raises((TypeError, ValueError), match=match):
            call(**kw)
    for kw, match in ((dict(ws=None), "WORKSPACE"), (dict(ws=ws[:16]), "WORKSPACE"), (dict(A=t["A"].float(), B=t["B"].float()), "ARG")):
        with pytest.raises((dg.DGError, ValueError), match=match + "|B holds|A holds"):
            call(**kw)
