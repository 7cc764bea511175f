"""Penalties, biases and masks in every form that the launch rule chooses: chunks of one, two and four groups a thread,
16-bit and 32-bit words of the table, histories shorter than their room (GPU).  Bit for bit, as in test_gpu_adjust."""
import numpy as np
import pytest

from tests.test_gpu_adjust import F, TYPES, draw, reference, run, same

pytestmark = pytest.mark.gpu


def expected(x, C, a):
    import torch
    return torch.from_numpy(reference(x.float().numpy(), C, a)).to(x.dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,room", [(300, 40000), (1, 50), (0, 7), (32767, 32770), (5, 5)])
def test_histories_of_a_wider_buffer(dg, dev, dtype, T, room):
    """T: the most tokens of a row; what lies behind them in the row's room does not count, whatever the lengths say."""
    x, a = draw((T, room), 3, 9001, 9004, room, 4, dtype)
    a["lens"] = np.array([T, max(T - 1, 0), room], np.int32)
    narrow = dict(a, tokens=a["tokens"][:, :T])
    same(run(dg, dev, x, 9001, a, T=T), expected(x, 9001, narrow), dtype)
    a["lens"] = narrow["lens"] = None
    same(run(dg, dev, x, 9001, a, T=T, in_place=True), expected(x, 9001, narrow), dtype)


def test_binding_refuses_more_tokens_than_a_row_has(dg, dev):
    import torch
    x, tok = torch.zeros(4, 100, device=dev), torch.zeros(4, 10, dtype=torch.int32, device=dev)
    for T in (11, -1):
        with pytest.raises(dg.DGError, match="DG_ERR_SHAPE"):
            dg.dg_adjust_rows(x, x, tokens=tok, T=T)
    with pytest.raises(ValueError, match="tokens holds"):     # the rows are as far apart as they are long
        dg.dg_adjust_rows(x, x, tokens=tok[:3], T=2)
