"""Sampling from given random numbers against the definition in 64 bits on the host (GPU).  Tokens are whole numbers
and have to be equal."""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

NEG = -np.inf
LARGEST_U = 1.0 - 2.0 ** -24


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def reference_row(x, u, T=1.0, k=0, p=1.0, mp=0.0):
    """x: float64 values of one row."""
    C = len(x)
    if np.isnan(x).any():
        return int(np.flatnonzero(np.isnan(x))[0])
    if not T > 0:
        return int(np.argmax(x))
    m = x.max()
    if m == NEG:
        return -1
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((x - m) / T)
    w[x == m] = 1.0
    w[~(w >= 0)] = 0.0
    w[w < 2.0 ** -(min(51, 62 - (C - 1).bit_length()) + 1)] = 0.0
    rank = np.argsort(-x, kind="stable")
    rank = rank[w[rank] > 0]
    if 0 < k < C:
        rank = rank[:k]
    if p < 1:
        sums = np.cumsum(w[rank].astype(np.longdouble))
        rank = rank[: min(len(rank), int(np.searchsorted(sums, np.longdouble(max(p, 0.0)) * sums[-1])) + 1)]
    if mp > 0:
        rank = rank[w[rank] >= min(mp, 1.0)]
    kept = np.sort(rank)
    sums = np.cumsum(w[kept].astype(np.longdouble))
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    at = int(np.searchsorted(sums, np.longdouble(u) * sums[-1], side="right"))
    return int(kept[min(at, len(kept) - 1)])


def sample(dg, dev, x, u, C=None, ws_fill=0xA5, **params):
    """x: CPU tensor [R][ld]; params: per-row lists or arrays (or absent)."""
    import torch
    R, ld = x.shape
    C = ld if C is None else C
    types = {"temperature": torch.float32, "top_k": torch.int32, "top_p": torch.float32, "min_p": torch.float32}
    given = {n: torch.tensor(np.asarray(v), dtype=types[n], device=dev) for n, v in params.items()}
    need = dg.dg_sample_workspace_bytes(R, C)
    ws = torch.full((need + 256,), ws_fill, dtype=torch.uint8, device=dev)
    idx = torch.full((R + 2,), -77, dtype=torch.int64, device=dev)
    dg.dg_sample_rows(x.to(dev), torch.tensor(np.asarray(u), dtype=torch.float32, device=dev), idx[1:R + 1], R=R, C=C,
                      ld=ld, ws=ws[:need] if need else None, **given)
    torch.cuda.synchronize()
    assert (ws[need:] == ws_fill).all(), "bytes behind the workspace changed"
    got = idx.cpu().numpy()
    assert got[0] == -77 and got[-1] == -77
    return got[1:-1]


def check(dg, dev, x, u, C=None, **params):
    got = sample(dg, dev, x, u, C=C, **params)
    C = x.shape[1] if C is None else C
    rows = x[:, :C].double().numpy()
    names = {"temperature": "T", "top_k": "k", "top_p": "p", "min_p": "mp"}
    import torch
    u32 = np.asarray(u, dtype=np.float32)
    for r in range(x.shape[0]):
        kw = {}
        for n, v in params.items():
            v = np.asarray(v)[r]
            kw[names[n]] = int(v) if n == "top_k" else float(np.float32(v))
        want = reference_row(rows[r].copy(), float(u32[r]), **kw)
        assert got[r] == want, f"row {r}: token {got[r]}, expected {want} ({kw}, u={u32[r]!r})"
    return got


def logits(key, R, ld, dtype, sigma):
    import torch
    return torch.from_numpy(synth.normal_f32(key, (R, ld), sigma)).to(tdtype(dtype))


SETS = {
    "plain": {},
    "temperature": {"temperature": (0.3, 0.7, 1.0, 1.6, 4.0, 0.05)},
    "top_k": {"top_k": (1, 2, 7, 50, 400, 3000)},
    "top_p": {"top_p": (0.1, 0.5, 0.9, 0.99, 0.9999, 0.02)},
    "min_p": {"min_p": (0.001, 0.02, 0.1, 0.3, 0.7, 1.0)},
    "top_k_top_p": {"top_k": (3, 40, 200, 1000, 2500, 60), "top_p": (0.9, 0.5, 0.95, 0.3, 0.99, 0.999)},
    "all": {"temperature": (0.5, 0.8, 1.0, 1.3, 2.0, 0.9), "top_k": (20, 50, 0, 1000, 64, 3),
            "top_p": (0.9, 1.0, 0.95, 0.8, 0.99, 0.7), "min_p": (0.05, 0.02, 0.1, 0.0, 0.01, 0.3)},
}


@pytest.mark.parametrize("C", [1, 2, 63, 65, 1000, 4096, 4097, 6144, 32003, 128256])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("which", sorted(SETS))
def test_definition(dg, dev, C, dtype, which):
    R, sigma = 6, (0.4, 2.0, 6.0)[C % 3]
    x = logits((1200, 1, C % 91, len(which)), R, C + 3, dtype, sigma)
    u = synth.uniform_f32((1201, 1, C % 91, len(which)), (R,), 0.0, LARGEST_U)
    check(dg, dev, x, u, C=C, **SETS[which])


@pytest.mark.parametrize("C", [300, 5000, 70001])
def test_many_equal_values(dg, dev, C):
    """Ties: the lowest indexes rank first, also where thousands share one value."""
    import torch
    rng = synth.rng(1210, 1, C % 7)
    x = torch.from_numpy(np.stack([
        np.zeros(C), np.full(C, -3.0), rng.integers(0, 2, C).astype(np.float64), rng.integers(0, 5, C) * 0.25,
        np.where(rng.random(C) < 0.9, 1.0, 0.5), rng.integers(-3, 3, C) * 1.0]).astype(np.float32))
    for u in (0.0, 0.3, 0.71, LARGEST_U):
        uu = [u] * 6
        check(dg, dev, x, uu)
        check(dg, dev, x, uu, top_k=[C // 2, C - 1, C // 3, 5, C // 2, 1])
        check(dg, dev, x, uu, top_p=[0.5, 0.25, 0.75, 0.6, 0.9, 0.3])
        check(dg, dev, x, uu, top_k=[C // 2, C - 1, C // 3, C // 4, C // 2, C // 5], top_p=[0.5, 0.25, 0.75, 0.6, 0.9, 0.3],
              min_p=[0.1, 0.9, 0.5, 0.8, 0.61, 0.2])


@pytest.mark.parametrize("C", [257, 9001])
def test_masked_rows(dg, dev, C):
    import torch
    x = logits((1220, 1, 0, 0), 8, C, "f32", 2.0)
    low = torch.finfo(torch.float32).min
    rng = synth.rng(1221, 1, 0)
    mask = torch.from_numpy(rng.random((8, C)) < 0.7)
    x[0][mask[0]] = NEG
    x[1][mask[1]] = low
    x[2] = NEG                        # nothing left
    x[3] = low                        # the lowest value everywhere: all alike
    x[4, 1:] = NEG                    # one token left
    x[4, 0] = -5.0
    x[5, :-1] = NEG
    x[6] = NEG
    x[6, C // 2] = low
    x[7][mask[7]] = NEG
    x[7][mask[0]] = low
    for params in ({}, {"top_k": [5] * 8}, {"top_p": [0.9] * 8}, {"min_p": [0.05] * 8},
                   {"top_k": [40] * 8, "top_p": [0.8] * 8, "temperature": [0.9] * 8}):
        got = check(dg, dev, x, [0.37] * 8, **params)
        assert got[2] == -1 and got[4] == 0 and got[5] == C - 1 and got[6] == C // 2
    got = check(dg, dev, x, [0.5] * 8, temperature=[0.0] * 8)
    assert got[2] == 0 and got[4] == 0


@pytest.mark.parametrize("C", [100, 6000])
def test_infinities_nan_and_extremes(dg, dev, C):
    import torch
    big = float(torch.finfo(torch.float32).max)
    x = logits((1230, 1, 0, 0), 8, C, "f32", 1.0)
    x[0, 7] = float("nan")
    x[0, 3] = float("inf")
    x[1, 20] = x[1, 50] = float("inf")
    x[2, 11] = big
    x[2, 12] = -big
    x[3, 4] = float("nan")
    x[4, 0] = 1e-40                   # subnormal among zeros
    x[4, 1:] = 0.0
    x[5] = torch.where(torch.arange(C) % 2 == 0, big, -big)
    x[6] = -big
    x[6, 9] = NEG
    x[7, 5] = NEG
    for T in (1.0, 0.01, 1e-30, 1e30, float("inf")):
        for params in ({}, {"top_k": [30] * 8}, {"top_p": [0.7] * 8}):
            got = check(dg, dev, x, [0.6] * 8, temperature=[T] * 8, **params)
            assert got[0] == 7 and got[3] == 4 and got[1] in (20, 50)


@pytest.mark.parametrize("C", [50, 5000])
def test_parameter_borders(dg, dev, C):
    x = logits((1240, 1, 0, 0), 10, C, "f32", 1.5)
    nan = float("nan")
    check(dg, dev, x, [0.0, LARGEST_U, 1.0, 1.5, -0.5, nan, 0.5, 2.0 ** -149, 0.25, 0.75])
    check(dg, dev, x, [0.4] * 10, top_k=[0, -1, C, C + 1, C - 1, 1, 2 ** 31 - 1, -2 ** 31, 2, 3])
    check(dg, dev, x, [0.4] * 10, top_p=[0.0, -1.0, 1.0, 2.0, nan, 1.0 - 2.0 ** -24, 1e-30, 0.5, 0.9, 0.1])
    check(dg, dev, x, [0.4] * 10, min_p=[0.0, -1.0, 1.0, 2.0, nan, 1e-30, 0.5, 0.9, 0.1, 1.0 - 2.0 ** -24])
    check(dg, dev, x, [0.4] * 10, temperature=[0.0, -1.0, nan, 1e-45, 1e38, 1.0, 0.5, 2.0, -0.0, 100.0])
    check(dg, dev, x, [LARGEST_U] * 10, top_k=[5] * 10, top_p=[0.0] * 10, min_p=[1.0] * 10)


@pytest.mark.parametrize("C", [37, 4500])
def test_shares_of_tokens(dg, dev, C):
    """With u at the midpoints of n equal steps, token c comes n * p(c) times, within one."""
    import torch
    n = 1500
    row = synth.normal_f32((1250, 1, 0, 0), (1, C), 2.0)
    x = torch.from_numpy(np.repeat(row, n, axis=0))
    u = (np.arange(n) + 0.5) / n
    got = sample(dg, dev, x, u, temperature=[1.3] * n, top_k=[30] * n)
    assert (np.diff(got) >= 0).all()
    w = np.exp((row[0].astype(np.float64) - row.max()) / np.float64(np.float32(1.3)))
    kept = np.argsort(-row[0], kind="stable")[:30]
    share = np.zeros(C)
    share[kept] = w[kept] / w[kept].sum()
    counts = np.bincount(got, minlength=C)
    assert (counts[share == 0] == 0).all()
    assert (np.abs(counts - n * share) <= 1.0 + 1e-6).all()


def test_more_rows_than_a_workspace_holds_at_once(dg, dev):
    R, C = 1100, 4100
    x = logits((1260, 1, 0, 0), R, C, "bf16", 2.0)
    u = synth.uniform_f32((1261, 1, 0, 0), (R,), 0.0, LARGEST_U)
    rng = synth.rng(1262, 1, 0)
    assert dg.dg_sample_workspace_bytes(R, C) == dg.dg_sample_workspace_bytes(512, C)
    check(dg, dev, x, u, temperature=rng.uniform(0.5, 1.5, R), top_k=rng.integers(0, 100, R),
          top_p=rng.uniform(0.5, 1.1, R), min_p=rng.uniform(-0.1, 0.1, R))


def test_more_rows_than_a_launch_has(dg, dev):
    import torch
    R, C = (1 << 21) + 5, 3
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(R, C, device=dev, generator=g)
    u = torch.rand(R, device=dev, generator=g)
    idx = torch.full((R,), -7, dtype=torch.int64, device=dev)
    dg.dg_sample_rows(x, u, idx)
    torch.cuda.synchronize()
    w = torch.exp(x.double() - x.double().amax(1, keepdim=True))
    cum = torch.cumsum(w, 1)
    assert torch.equal(idx, (cum <= u.double().unsqueeze(1) * cum[:, -1:]).sum(1))


def test_a_row_does_not_depend_on_its_batch(dg, dev):
    R, C = 40, 20011
    x = logits((1270, 1, 0, 0), R, C, "f16", 3.0)
    u = synth.uniform_f32((1271, 1, 0, 0), (R,), 0.0, LARGEST_U)
    p = {"temperature": [0.8] * R, "top_k": [100] * R, "top_p": [0.9] * R}
    whole = sample(dg, dev, x, u, ws_fill=0xFF, **p)
    for r in (0, 17, 39):
        one = sample(dg, dev, x[r:r + 1], u[r:r + 1], ws_fill=0, **{n: v[:1] for n, v in p.items()})
        assert one[0] == whole[r]
    assert np.array_equal(whole, sample(dg, dev, x, u, **p))


def test_long_row(dg, dev):
    """Sub-chunks longer than the shortest (rows past two million)."""
    C = 3_000_017
    x = logits((1280, 1, 0, 0), 1, C, "f32", 1.0)
    check(dg, dev, x, [0.7])
    check(dg, dev, x, [0.7], top_p=[0.9])
    check(dg, dev, x, [0.2], top_k=[100000], top_p=[0.5])


def test_greedy_equals_argmax(dg, dev):
    import torch
    vals, _ = synth.argmax_logits(1290, 8, 50003)
    x = torch.from_numpy(vals)
    got = sample(dg, dev, x, [0.5] * 8, temperature=[0.0] * 8, top_k=[5] * 8, top_p=[0.5] * 8)
    idx = torch.zeros(8, dtype=torch.int64, device=dev)
    ws = torch.zeros(dg.dg_argmax_workspace_bytes(8, 50003), dtype=torch.uint8, device=dev)
    dg.dg_argmax_rows(x.to(dev), idx, ws=ws)
    torch.cuda.synchronize()
    assert np.array_equal(got, idx.cpu().numpy())


def test_graph_replays(dg, dev):
    """A captured call, with new logits, numbers and parameters between replays, against eager calls."""
    import torch
    R, C = 6, 33000
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn(R, C, device=dev, generator=g)
    u = torch.rand(R, device=dev, generator=g)
    T, p = torch.ones(R, device=dev), torch.full((R,), 0.9, device=dev)
    k = torch.full((R,), 50, dtype=torch.int32, device=dev)
    idx = torch.zeros(R, dtype=torch.int64, device=dev)
    ws = torch.zeros(dg.dg_sample_workspace_bytes(R, C), dtype=torch.uint8, device=dev)

    def step():
        dg.dg_sample_rows(x, u, idx, temperature=T, top_k=k, top_p=p, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        x.copy_(torch.randn(R, C, device=dev, generator=g) * (rep + 1))
        u.copy_(torch.rand(R, device=dev, generator=g))
        k.fill_(rep * 37)
        p.fill_(0.5 + 0.2 * rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = idx.clone()
        idx.fill_(-5)
        ws.fill_(0xA5)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, idx)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 300, 512, 513, 1000, 1023, 1024, 1025, 2500, 4097])
def test_border_lists_of_every_length(dg, dev, n):
    """n tokens share one bin, equal or a few steps apart, and every border falls among them."""
    import torch
    C = 9001
    g = np.random.default_rng(n)
    rows, par = [], {"temperature": [], "top_k": [], "top_p": [], "min_p": []}
    for steps in (0, 1, 5):   # distinct values of the bin
        for k, p, mp in ((n // 2 + 1, 1.0, 0.0), (0, 0.37, 0.0), (n // 3 + 1, 0.61, 0.0), (n, 0.999, 0.5), (0, 0.0, 0.0)):
            v = np.full(C, -np.inf, np.float32)
            at = g.permutation(C)[:n]
            v[at] = np.float32(3.0) + np.float32(2.0 ** -20) * g.integers(0, steps + 1, n).astype(np.float32)
            v[g.permutation(C)[:50]] = -60.0   # a long range, so that the values above share a bin
            v[at] = np.maximum(v[at], np.float32(3.0))
            rows.append(v)
            for name, value in zip(("temperature", "top_k", "top_p", "min_p"), (1.0, k, p, mp)):
                par[name].append(value)
    check(dg, dev, torch.from_numpy(np.stack(rows)), g.random(len(rows)), **par)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ld", [33000, 33001])   # rows aligned for wide loads, and not
def test_extremes_of_chunks_of_several_steps(dg, dev, dtype, ld):
    """So many rows that a workgroup takes several load steps: NaN, equal maxima, zeros of both signs, masked rows."""
    import torch
    R, C = 90, 32999
    x = logits((1295, 1, 0, 0), R, ld, dtype, 2.0)
    x[:, C:] = float("nan")   # behind the rows, never read
    g = np.random.default_rng(5)
    want = []
    for r in range(R):
        spots = np.sort(g.choice(C, 3, replace=False))
        kind = r % 9
        if kind == 0:
            x[r, spots] = 20.0
        elif kind == 1:
            x[r, spots] = float("nan")
        elif kind == 2:
            x[r, :C] = -float("inf")
        elif kind == 3:
            x[r, :C] = -float("inf")
            x[r, spots] = 1.0
        elif kind == 4:
            x[r, :C] = -x[r, :C].abs() - 1
            x[r, spots] = 0.0
            x[r, spots[0]] = -0.0
        elif kind == 5:
            x[r, :C] = -7.0
        elif kind == 6:
            x[r, spots[1:]] = float("inf")
            x[r, spots[0]] = -float("inf")
        elif kind == 7:
            x[r, 0], x[r, C - 1] = 30.0, 30.0
        row = x[r, :C].double().numpy()
        want.append(int(np.flatnonzero(np.isnan(row))[0]) if np.isnan(row).any() else int(row.argmax()))
    got = sample(dg, dev, x, [0.3] * R, C=C, temperature=[0.0] * R)
    assert np.array_equal(got, want)
    draws = x.clone()
    keep = [r for r in range(R) if r % 9 not in (1, 2)]
    many = torch.cat([draws[keep], draws[keep][:20]])   # still so many rows
    n = many.shape[0]
    check(dg, dev, many, g.random(n), C=C, temperature=[0.9] * n, top_k=[60] * n, top_p=[0.95] * n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,ld", [(4097, 4104), (6145, 6152), (9001, 9001 + 2048), (33001, 33008)])
def test_nothing_behind_a_row_is_listed(dg, dev, C, ld, dtype):
    """Rows of one value, of one allowed token, of a few tied ones, and rows whose spread overflows binary32: what is
    behind a row is neither drawn nor listed (no key of its value in the workspace)."""
    import torch
    behind = 12352.0   # exact in every type
    R = 8
    x = torch.full((R, ld), behind, dtype=torch.float32)
    x[0, :C] = 1.0
    x[1, :C] = NEG
    x[1, C // 3] = -2.0
    x[2, :C] = NEG
    x[2, 7::C // 5] = 0.5
    x[3, :C] = torch.where(torch.arange(C) % 2 == 0, 3e38, -3e38)
    x[4, :C] = torch.finfo(torch.float32).min / 2
    x[5, :C] = NEG
    x[5, C - 1] = 3.0
    x[6, :C] = NEG
    x[6, :20] = -1.0
    x[7, :C] = 1.0
    x[:, C:] = behind
    x = x.to(tdtype(dtype))
    spread = [1.0, 1.0, 0.7, float("inf"), 2.0, 1.0, 1.5, 1e38]
    for params in ({"top_p": [0.9] * R}, {"top_k": [3] * R}, {"top_k": [4] * R, "top_p": [0.6] * R, "min_p": [0.5] * R}):
        want = []
        for r in range(R):
            kw = {n: v[r] for n, v in params.items()}
            want.append(reference_row(x[r, :C].double().numpy(), float(np.float32(0.55)), T=float(np.float32(spread[r])),
                                      k=kw.get("top_k", 0), p=float(np.float32(kw.get("top_p", 1.0))),
                                      mp=kw.get("min_p", 0.0)))
        ws = torch.full((dg.dg_sample_workspace_bytes(R, C),), 0xA5, dtype=torch.uint8, device=dev)
        idx = torch.zeros(R, dtype=torch.int64, device=dev)
        given = {n: torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32, device=dev)
                 for n, v in params.items()}
        dg.dg_sample_rows(x.to(dev), torch.full((R,), 0.55, device=dev), idx, R=R, C=C, ld=ld, ws=ws,
                          temperature=torch.tensor(spread, device=dev), **given)
        torch.cuda.synchronize()
        assert idx.cpu().tolist() == want
        image = int(np.float32(behind).view(np.uint32)) | 0x80000000   # the upper half of its keys
        words = ws.cpu().numpy().view(np.uint32)
        assert not (words == image).any()
