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


# 512 and 1024 chunks of one group a thread (4096 binary32 logits, 8192 of 16 bits) are where chunks of two and four
# begin; in the last chunk of a row a few logits, and the whole of it; words of the mask that end inside a chunk
FORMS = [("f32", 128, 16384, 16384, 40, 3), ("f32", 75, 32003, 32011, 300, 40), ("f32", 130, 16387, 16388, 0, 9),
         ("f32", 256, 16384, 16391, 100, 0), ("f32", 150, 32003, 32004, 4000, 40), ("f32", 200, 49157, 49157, 70, 300),
         ("f16", 128, 32768, 32768, 40, 3), ("f16", 150, 32003, 32011, 1000, 8), ("bf16", 130, 32777, 32779, 300, 40),
         ("bf16", 256, 32768, 32771, 100, 0), ("f16", 260, 32777, 32777, 4000, 300), ("bf16", 206, 65539, 65540, 0, 40),
         ("bf16", 260, 32777, 32784, 32767, 5)]


@pytest.mark.parametrize("dtype,R,C,ld,T,B", FORMS)
def test_chunks_of_several_groups(dg, dev, dtype, R, C, ld, T, B):
    for mask in (False, True):
        x, a = draw((R, C, T, B, mask), R, C, ld, T, B, dtype, mask)
        want = expected(x, C, a)
        same(run(dg, dev, x, C, a, ldy=C + 3), want, dtype)
        same(run(dg, dev, x, C, a, in_place=True), want, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C,T,B", [(3, 20003, 32768, 9), (3, 20003, 70001, 0), (130, 32003, 32768, 40), (260, 32777, 33001, 5)])
def test_long_histories(dg, dev, dtype, R, C, T, B):
    """More tokens than a 16-bit count holds: words of 32 bits at every width of a chunk that 16-bit logits have."""
    x, a = draw((R, T), R, C, C + 1, T, B, dtype)
    want = expected(x, C, a)
    same(run(dg, dev, x, C, a), want, dtype)
    same(run(dg, dev, x, C, a, in_place=True), want, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [32766, 32767, 32768, 100003])
def test_one_token_throughout(dg, dev, dtype, T):
    """Every token of a history the same, prompt and output: the largest count beside neighbours that have none, that have
    all but one, and that are in the prompt alone."""
    C = 9000
    tok = np.full((6, T), 8190, np.int32)
    tok[1], tok[2, 0], tok[3, 1:], tok[4, : T // 2], tok[5] = 8191, 8191, 8191, 8191, C - 1
    a = dict(tokens=tok, prompt_lens=np.array([0, 0, 1, 1, T // 2, T - 1], np.int32), frequency=np.full(6, 2.0 ** -13, F),
             presence=np.full(6, 0.5, F), repetition=np.full(6, 1.25, F))
    import torch
    x = torch.from_numpy(np.random.default_rng(T).standard_normal((6, C)).astype(F)).to(getattr(torch, {
        "f32": "float32", "f16": "float16", "bf16": "bfloat16"}[dtype]))
    same(run(dg, dev, x, C, a), expected(x, C, a), dtype)
