"""The gated feed-forward products against their definition in 64 bits on the stored codes (GPU).

Tolerance, derived per output: a sum of K/32 block terms (each exact up to the
one rounding of its addition) through at most K/32 + 16 additions is off by at
most (K/32 + 16) 2^-24 sum|terms|; the activations are Lipschitz with a
constant below 1.2 and are evaluated to a relative error of (8 + 4 |z|) 2^-24,
z the argument of the exponential; the product adds one rounding.
"""
import math

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "gelu_tanh", "relu")
STEP = 2.0 ** -24


def decode(fmt, W, N, K):
    """(scales [N][K/32], codes [N][K/32][32]) in float64 from row-major bytes."""
    b = np.ascontiguousarray(W).reshape(N, K // 32, 18 if fmt == "q4_0" else 34)
    d = b[..., :2].copy().view(np.float16).astype(np.float64)[..., 0]
    if fmt == "q4_0":
        q = np.concatenate([b[..., 2:] & 15, b[..., 2:] >> 4], axis=-1).astype(np.float64) - 8
    else:
        q = b[..., 2:].copy().view(np.int8).astype(np.float64)
    return d, q


def columns(Xq, M, K):
    b = np.ascontiguousarray(Xq).reshape(M, K // 32, 36)
    return b[..., :2].copy().view(np.float16).astype(np.float64)[..., 0], b[..., 4:].copy().view(np.int8).astype(np.float64)


def sums(fmt, W, Xq, N, K, M):
    """(exact sums [M][N], sums of the terms' magnitudes)."""
    d, q = decode(fmt, W, N, K)
    dx, qx = columns(Xq, M, K)
    s, a = np.zeros((M, N)), np.zeros((M, N))
    for b in range(K // 32):
        t = (qx[:, b] @ q[:, b].T) * np.outer(dx[:, b], d[:, b])
        s += t
        a += np.abs(t)
    return s, a


def act64(name, g):
    """(act(g), |argument of the exponential|)."""
    if name == "silu":
        return g / (1 + np.exp(-g)), np.abs(g)
    if name == "gelu":
        return 0.5 * g * np.vectorize(math.erfc)(-g * math.sqrt(0.5)), g * g / 2
    if name == "gelu_tanh":
        z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        return g / (1 + np.exp(-z)), np.abs(z)
    return np.maximum(g, 0), np.zeros_like(g)


def check(name, Y, G, U, K):
    g, ga = G
    u, ua = U
    n = (K // 32 + 16) * STEP
    with np.errstate(over="ignore"):
        a, z = act64(name, g)
    dg, du = n * ga, n * ua
    tol = 1.2 * dg * (np.abs(u) + du) + np.abs(a) * du + (9 + 4 * z) * STEP * np.abs(a * u) * 1.01 + 2.0 ** -126
    err = np.abs(Y.astype(np.float64) - a * u)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), f"{name} at {worst}: got {Y[worst]!r}, expected {(a * u)[worst]!r}, tolerance {tol[worst]:.3e}"


def operands(orc, fmt, key, N, K, M, spread=1.0):
    quant = orc.quantize_q4_0 if fmt == "q4_0" else orc.quantize_q8_0
    Wg = quant(synth.normal_f32((key, 0, 0, 0), (N, K), spread / math.sqrt(K)))
    Wu = quant(synth.normal_f32((key, 0, 1, 0), (N, K), 1.0 / math.sqrt(K)))
    Xq = orc.quantize_q8_1(synth.normal_f32((key, 1, 0, 0), (M, K), 1.5))
    return Wg, Wu, Xq


def dev_u8(dev, a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).reshape(-1).view(np.uint8)).to(dev)


class Case:
    """One shape's operands on the device, both layouts, and the exact sums."""

    def __init__(self, dg, dev, orc, fmt, key, N, K, M, spread=2.0):
        import torch
        self.dg, self.dev, self.fmt, self.N, self.K, self.M = dg, dev, fmt, N, K, M
        self.Wg, self.Wu, self.Xq = operands(orc, fmt, key, N, K, M, spread)
        self.G = sums(fmt, self.Wg, self.Xq, N, K, M)
        self.U = sums(fmt, self.Wu, self.Xq, N, K, M)
        self.x = dev_u8(dev, self.Xq)
        self.rows = [dev_u8(dev, self.Wg), dev_u8(dev, self.Wu)]
        nbytes = getattr(dg, f"dg_{fmt}_tiles_bytes")(N, K)
        self.tiles = [torch.empty(nbytes, dtype=torch.uint8, device=dev) for _ in range(2)]
        for w, t in zip(self.rows, self.tiles):
            getattr(dg, f"dg_repack_{fmt}_tiles")(w, t, N, K)

    def run(self, tiles, act, same=False):
        import torch
        guard = 1024
        buf = torch.full((2 * guard + self.M * self.N,), -77.0, device=self.dev)
        Y = buf[guard:guard + self.M * self.N]
        wg, wu = self.tiles if tiles else self.rows
        if same:
            wu = wg
        if tiles:
            getattr(self.dg, f"dg_gemv_{self.fmt}_tiles_glu")(wg, wu, self.x, Y, self.N, self.K, self.M, act=act)
        else:
            getattr(self.dg, f"dg_gemv_{self.fmt}_glu")(wg, wu, self.x, Y, self.N, self.K, self.M, act=act)
        torch.cuda.synchronize()
        assert (buf[:guard] == -77).all() and (buf[-guard:] == -77).all(), "wrote outside Y"
        return Y.cpu().numpy().reshape(self.M, self.N)


# row-major: units of one to four (M * units <= 8), matrix cores at every padded column count; rows not a multiple of
# any tile; K of an odd number of 256s and past four units
SHAPES = [(1, 256, 1), (15, 256, 4), (16, 512, 24), (17, 768, 17), (300, 4096, 1), (129, 4096, 2), (65, 4352, 3),
          (40, 4096, 4), (33, 8448, 2), (70, 8192, 4), (8200, 512, 6), (8195, 512, 20), (4200, 768, 7), (4100, 4352, 17), (23, 4096, 5), (25, 4096, 6), (50, 16384, 2), (31, 16384, 3), (20, 16640, 1), (45, 2048, 5),
          (37, 2304, 8), (64, 4096, 9), (100, 1280, 16), (81, 4608, 17), (95, 2560, 18), (48, 4096, 24)]


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("N,K,M", SHAPES)
def test_definition(dg, dev, orc, fmt, N, K, M):
    c = Case(dg, dev, orc, fmt, 1300 + M, N, K, M)
    act = ACTS[(N + M) % 4]
    for tiles in (False, True):
        Y = c.run(tiles, act)
        check(act, Y, c.G, c.U, K)
        assert np.array_equal(Y, c.run(tiles, act)), "not reproducible"


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("M", range(1, 25))
def test_every_column_count(dg, dev, orc, fmt, M):
    N, K = 83, 1024
    c = Case(dg, dev, orc, fmt, 1340, N, K, M)
    for tiles in (False, True):
        check("silu", c.run(tiles, "silu"), c.G, c.U, K)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 6])
def test_activations_over_a_wide_range(dg, dev, orc, act, M):
    """Gates from far below to far above zero (spread 40), and a matrix gated by itself."""
    N, K = 200, 512
    c = Case(dg, dev, orc, "q8_0", 1350, N, K, M, spread=40.0)
    assert c.G[0].min() < -60 and c.G[0].max() > 60
    for tiles in (False, True):
        check(act, c.run(tiles, act), c.G, c.U, K)
        check(act, c.run(tiles, act, same=True), c.G, c.G, K)


# tiled: every shape of workgroup, column slices, columns in several passes (of unequal lengths too)
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("N,K,M", [(40, 28672, 24), (100, 20480, 24), (33, 65536, 9), (17, 81920, 1), (1024, 2048, 12),
                                   (2100, 512, 24), (2100, 6912, 17), (5130, 512, 8), (5130, 512, 16), (5200, 256, 20),
                                   (5130, 5888, 24), (8200, 512, 3), (9000, 256, 16), (8192, 3328, 24), (16400, 256, 2),
                                   (16385, 512, 12), (16384, 3328, 24), (16390, 2816, 8)])
def test_tiled_launch_shapes(dg, dev, orc, fmt, N, K, M):
    c = Case(dg, dev, orc, fmt, 1360, N, K, M)
    check("silu", c.run(True, "silu"), c.G, c.U, K)


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_columns_do_not_depend_on_the_other_columns(dg, dev, orc, fmt):
    """A NaN in one column stays in it (columns past M re-read others, whose results are dropped)."""
    N, K, M = 50, 512, 11
    c = Case(dg, dev, orc, fmt, 1380, N, K, M)
    clean = [c.run(t, "silu") for t in (False, True)]
    bad = c.Xq.copy().reshape(M, K // 32, 36)
    bad[M - 1, 0, :2] = np.array([np.nan], dtype=np.float16).view(np.uint8)
    c.x = dev_u8(dev, bad)
    for t in (False, True):
        y = c.run(t, "silu")
        assert np.array_equal(y[:M - 1], clean[t][:M - 1]) and np.isnan(y[M - 1]).all()


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("M", [1, 3])
def test_matrices_past_four_gibibytes(dg, dev, tiles, M):
    import torch
    N, K = (262161, 16384) if M == 1 else (131077, 32768)   # rows in units, matrix cores
    nb, T = K // 32, -(-N // 16)
    g = torch.Generator(device=dev).manual_seed(7)
    size = T * (K // 256) * 4352 if tiles else N * nb * 34
    assert size > 1 << 32
    # zero bytes but for the last 16-row tile's rows, whose blocks are random
    W = [torch.zeros(size, dtype=torch.uint8, device=dev) for _ in range(2)]
    first = (T - 1) * 16
    n = N - first
    rows = []
    for w in W:
        q = torch.randint(-50, 51, (n, nb, 32), device=dev, generator=g, dtype=torch.int8)
        d = (torch.rand(n, nb, 1, device=dev, generator=g) * 1e-3).half()
        b = torch.cat([d.view(torch.uint8), q.view(torch.uint8)], -1).contiguous()
        if tiles:
            t = torch.empty(dg.dg_q8_0_tiles_bytes(n, K), dtype=torch.uint8, device=dev)
            dg.dg_repack_q8_0_tiles(b.reshape(-1), t, n, K)
            w[-t.numel():] = t
        else:
            w[-b.numel():] = b.reshape(-1)
        rows.append(b.cpu().numpy())
    Xq = torch.empty(M * nb * 36, dtype=torch.uint8, device=dev)
    dg.dg_quantize_q8_1(torch.randn(M, K, device=dev, generator=g), Xq, M, K)
    Y = torch.full((M, N), 5.0, device=dev)
    if tiles:
        dg.dg_gemv_q8_0_tiles_glu(W[0], W[1], Xq, Y, N, K, M)
    else:
        dg.dg_gemv_q8_0_glu(W[0], W[1], Xq, Y, N, K, M)
    torch.cuda.synchronize()
    assert not Y[:, :first].any()
    x = Xq.cpu().numpy()
    G, U = (sums("q8_0", r, x, n, K, M) for r in rows)
    check("silu", Y[:, first:].cpu().numpy(), G, U, K)


def test_empty(dg, dev):
    import torch
    w = torch.zeros(4096, dtype=torch.uint8, device=dev)
    y = torch.full((3, 4), 2.0, device=dev)
    dg.dg_gemv_q4_0_glu(w, w, w, y, 4, 256, 0)
    dg.dg_gemv_q4_0_glu(w, w, w, y, 0, 256, 3)
    torch.cuda.synchronize()
    assert (y == 2.0).all()
    dg.dg_gemv_q4_0_glu(w, w, w, y, 4, 0, 3)   # empty sums
    torch.cuda.synchronize()
    assert (y == 0.0).all()
    y.fill_(2.0)
    dg.dg_gemv_q8_0_tiles_glu(w, w, w, y, 4, 0, 3)
    torch.cuda.synchronize()
    assert (y == 0.0).all()


def test_empty_sums_past_two_to_the_32(dg, dev):
    """More outputs than one launch has threads."""
    import torch
    N, M = 1 << 28, 17
    Y = torch.ones(M, N, dtype=torch.float32, device=dev)
    none = torch.zeros(16, dtype=torch.uint8, device=dev)
    dg.dg_gemv_q4_0_tiles_glu(none, none, none, Y, N, 0, M)
    for m in range(M):
        assert torch.count_nonzero(Y[m]).item() == 0


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("N,K,M", [(200003, 256, 1), (197001, 512, 3), (132100, 256, 5)])
def test_more_rows_than_a_wave_holds_outputs(dg, dev, orc, fmt, N, K, M):
    """Past 64 rows a wave stores a full set of outputs and goes on."""
    c = Case(dg, dev, orc, fmt, 1390, N, K, M)
    check("silu", c.run(False, "silu"), c.G, c.U, K)


@pytest.mark.parametrize("tiles,M", [(True, 9), (True, 3), (False, 9)])
def test_rows_past_a_launch(dg, dev, tiles, M):
    """More rows than the threads of one launch reach (eight a row), in several or in several row groups a workgroup."""
    import torch
    N, K = (1 << 29) + 37, 256
    nb, row = K // 32, 18 * (K // 32)   # also a tile's bytes a row: one group of K
    g = torch.Generator(device=dev).manual_seed(9)
    W = torch.zeros(-(-N // 16) * 16 * row, dtype=torch.uint8, device=dev)   # gate and up; zero but for these rows
    spots = [0, (1 << 26) - 32, (1 << 27) - 16, (1 << 28) - 16, (1 << 29) - 16]
    some = []
    for first in spots:
        n = min(64, N - first)
        q = torch.empty(n * row, dtype=torch.uint8, device=dev)
        dg.dg_quantize_q4_0(torch.randn(n, K, device=dev, generator=g) / 16, q, n, K)
        some.append((first, n, q.cpu().numpy()))
        if tiles:
            t = torch.empty(dg.dg_q4_0_tiles_bytes(n, K), dtype=torch.uint8, device=dev)
            dg.dg_repack_q4_0_tiles(q, t, n, K)
            W[first * row:first * row + t.numel()] = t
        else:
            W[first * row:first * row + q.numel()] = q
    Xq = torch.empty(M * nb * 36, dtype=torch.uint8, device=dev)
    dg.dg_quantize_q8_1(torch.randn(M, K, device=dev, generator=g), Xq, M, K)
    Y = torch.full((M, N), 5.0, device=dev)
    (dg.dg_gemv_q4_0_tiles_glu if tiles else dg.dg_gemv_q4_0_glu)(W, W, Xq, Y, N, K, M)
    torch.cuda.synchronize()
    x = Xq.cpu().numpy()
    for first, n, q in some:
        G = sums("q4_0", q, x, n, K, M)
        check("silu", Y[:, first:first + n].cpu().numpy(), G, G, K)
        Y[:, first:first + n] = 0
    for m in range(M):   # and every other row was written, with zeros
        assert torch.count_nonzero(Y[m]).item() == 0
