"""Low-rank adapters at the sizes that fill the machine, whose workgroups take 512 outputs, in every kernel (GPU).  The
definition and its tolerance are test_gpu_lora's."""
import numpy as np
import pytest

from tests.test_gpu_lora import TYPES, Case

pytestmark = pytest.mark.gpu

# (M, N, R, L) with 1024 workgroups of 512 outputs and more: windows of four rows of one adapter, of several adapters,
# and workgroups for rows where a window has fewer than there are adapters; outputs that end in a block's first and last
SHAPES = [(1100, 777, 8, 1), (1100, 1024, 16, 1), (1101, 769, 32, 1), (1030, 1025, 64, 1), (1100, 600, 128, 1),
          (1100, 513, 256, 1), (1060, 700, 512, 1), (300, 5121, 24, 9), (200, 8705, 32, 64), (200, 2561, 40, 300)]


@pytest.mark.parametrize("w", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,R,L", SHAPES)
def test_blocks_of_512(dg, dev, M, N, R, L, w):
    x = TYPES[(M + N + R) % 3]
    ranks = np.random.default_rng(R).integers(0, R + 2, L) if L > 1 else None
    adapter = np.random.default_rng(M).integers(-1, L, M)
    c = Case((M, N, R), M, N, 72, R, L, x, w, ranks=ranks, adapter=adapter)
    got = c.check(dg, dev)
    assert np.array_equal(got, c.run(dg, dev, in_place=True, fill=0xFF))
    for m in (0, M // 2, M - 1):      # a row alone: blocks of 256, or one launch
        one = Case((M, N, R), M, N, 72, R, L, x, w, ranks=ranks, adapter=adapter)
        one.M, one.x, one.adapter, one.base = 1, c.x[m:m + 1], c.adapter[m:m + 1], c.base[m:m + 1]
        assert np.array_equal(one.run(dg, dev)[0], got[m])
