"""Routed experts in every kernel that the launch rules choose, at the sizes that choose them (GPU).

Definitions and tolerances are those of test_gpu_moe; weights are quantised on the device, and the bytes that the library
reads are the ones that the definition decodes."""
import math

import numpy as np
import pytest

from tests.test_gpu_moe import Layer, distinct

pytestmark = pytest.mark.gpu

BLOCK = {"q4_0": 18, "q8_0": 34}


class Large(Layer):
    """A Layer whose weights are made on the device."""

    def __init__(self, dg, dev, orc, fmt, key, E, N, K, M, ids, act="silu"):
        import synth
        import torch
        self.dg, self.dev, self.fmt, self.E, self.N, self.K, self.M, self.act = dg, dev, fmt, E, N, K, M, act
        self.ids = np.asarray(ids, np.int32).reshape(M, -1)
        self.k = self.ids.shape[1]
        self.rows, self.tiles = {}, {}
        g = torch.Generator(device=dev).manual_seed(key)
        for n, r, c, s in (("Wg", N, K, 2.0), ("Wu", N, K, 1.0), ("Wd", K, N, 1.0)):
            w = torch.empty(E * r * (c // 32) * BLOCK[fmt], dtype=torch.uint8, device=dev)
            getattr(dg, f"dg_quantize_{fmt}")(torch.randn(E * r, c, device=dev, generator=g) * (s / math.sqrt(c)), w, E * r, c)
            t = torch.empty(getattr(dg, f"dg_{fmt}_tiles_bytes")(E * r, c), dtype=torch.uint8, device=dev)
            self.tiles[n] = getattr(dg, f"dg_repack_{fmt}_tiles")(w, t, E * r, c)
            self.rows[n] = w.cpu().numpy().reshape(E, -1)
        self.Xq = np.ascontiguousarray(orc.quantize_q8_1(synth.normal_f32((key, 1, 0, 0), (M, K), 1.5))).reshape(M, -1)
        self.w = np.random.default_rng(key).random((M, self.k)).astype(np.float32) - np.float32(0.2)


# What each (E, N, K, M, k) is for, on 256 compute units.  Gated products: eight waves (K > 2048 and 256 workgroups of 64
# rows) with up to 8 tokens and with more; four waves that take several row groups each, up to 8 tokens.  Down products:
# two parts of K (N >= 4096) where the tokens' own weights would be read too often, up to 8 tokens and more; one part,
# several row groups, up to 8 tokens; a token's products and sum in one kernel with one, two and four row tiles a
# workgroup, in one part of K and two, and the most waves that it takes.
FORMS = {
    "q4_0": [(4, 4096, 2304, 2, 2), (2, 8448, 2304, 8, 2), (2, 8448, 2560, 11, 2), (20, 2304, 256, 8, 20), (2, 4608, 768, 8, 2),
             (2, 4608, 768, 18, 2), (20, 256, 4608, 8, 20), (4, 256, 4352, 2, 2), (4, 256, 4352, 8, 2), (4, 768, 4096, 2, 4),
             (3, 4096, 512, 3, 2), (2, 4096, 4096, 2, 2), (4, 4096, 2048, 8, 1), (8, 4096, 256, 5, 8), (16, 256, 512, 5, 16)],
    "q8_0": [(4, 4096, 2304, 2, 2), (2, 8448, 2304, 8, 2), (2, 8448, 2560, 11, 2), (2, 4608, 768, 8, 2),
             (2, 4608, 768, 18, 2), (20, 256, 4608, 8, 20), (4, 256, 4352, 2, 2), (4, 256, 4352, 8, 2), (4, 768, 4096, 2, 4),
             (3, 4096, 512, 3, 2), (4, 4096, 1024, 8, 1), (9, 4096, 2048, 8, 1), (8, 4096, 256, 5, 8), (16, 256, 512, 5, 16)]}
CASES = [(f, *s) for f in FORMS for s in FORMS[f]]


@pytest.mark.parametrize("fmt,E,N,K,M,k", CASES)
def test_definition_and_independence(dg, dev, orc, fmt, E, N, K, M, k):
    """The definition, and each token of the batch the bits that it has alone, with one other, and without some."""
    c = Large(dg, dev, orc, fmt, 3100 + E + N + M, E, N, K, M, distinct((E, N, K), E, M, k), act=("silu", "gelu_tanh")[M % 2])
    Y, H = c.check()
    for rows in [[m] for m in range(M)] + [[M - 1, 0], list(range(1, M)), list(range(M))[::-1]]:
        if not rows:
            continue
        Y1, H1 = c.run(rows=rows, fill=0)
        assert np.array_equal(Y1, Y[rows]) and np.array_equal(H1, H[rows]), rows


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("E,N,K,M,k", [(4, 4096, 2304, 3, 2), (2, 4608, 768, 8, 2), (20, 256, 4608, 8, 20), (4, 4096, 1024, 8, 1)])
def test_slots_without_experts(dg, dev, orc, fmt, E, N, K, M, k):
    """Absent and repeated experts, ids outside the range, a token without any, NaN in what does not count."""
    ids = distinct((E, M), E, M, k)
    ids[0] = -1
    ids[1, 0], ids[2] = E, ids[2, 0]
    c = Large(dg, dev, orc, fmt, 3300 + E, E, N, K, M, ids)
    Y, _ = c.check("bf16")
    assert not Y[0].any()
    c.w[(c.ids < 0) | (c.ids >= E)] = np.nan
    assert np.array_equal(Y, c.run("bf16", fill=0xFF)[0])


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("E,N,K,M,k", [(2, 4608, 768, 18, 2), (20, 256, 4608, 8, 20), (4, 4096, 1024, 8, 1)])
def test_types_of_the_weighted_sum(dg, dev, orc, fmt, E, N, K, M, k):
    """16-bit outputs are one rounding of the binary32 sums, made by a launch of their own and beside the down products."""
    import torch
    c = Large(dg, dev, orc, fmt, 3500 + E, E, N, K, M, distinct((E, M, 1), E, M, k))
    Y, H = c.check()
    for out, t in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        Y16, H16 = c.run(out)
        assert np.array_equal(Y16, torch.from_numpy(Y).to(t).float().numpy()) and np.array_equal(H, H16)
