"""The operators of a batch of different requests where a call is more than one launch of each kernel: 2^21 workgroups
and more (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

MOST = 1 << 21   # workgroups of a launch


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router(dg, dev, score):
    """Four tokens a workgroup."""
    import torch
    M = 4 * MOST + 7
    x = torch.randn(M, 3, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
    ids, w = torch.full((M, 2), -9, dtype=torch.int32, device=dev), torch.full((M, 2), -9.0, device=dev)
    dg.dg_moe_route(x, ids, w, score=score, renorm=False)
    s = x.double()
    s = torch.softmax(s, 1) if score == "softmax" else torch.sigmoid(s)
    v, order = torch.sort(s, dim=1, descending=True, stable=True)
    torch.cuda.synchronize()
    assert torch.equal(ids, order[:, :2].int())
    assert ((w - v[:, :2]).abs() <= 2.0 ** -24 * (1 + 2.0 ** -20) * v[:, :2]).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_adjustments(dg, dev, dtype):
    """A row a workgroup."""
    import torch
    R = MOST + 5
    x = torch.randn(R, 3, device=dev, generator=torch.Generator(device=dev).manual_seed(2)).to(getattr(torch, dtype))
    tok = (torch.arange(R, device=dev, dtype=torch.int32) * 7 % 4).view(R, 1)   # 3: none
    rep, y = torch.full((R,), 2.0, device=dev), torch.zeros_like(x)
    dg.dg_adjust_rows(x, y, tokens=tok, repetition=rep)
    want = torch.where(tok == torch.arange(3, device=dev), torch.where(x > 0, x / 2, x * 2), x)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_adapters(dg, dev):
    """256 rows and 8192 blocks of outputs a launch: the outputs behind them, with an adapter and without."""
    import torch
    M, N, K, R, L = 256, 8192 * 512 + 77, 8, 8, 256
    g = torch.Generator(device=dev).manual_seed(3)
    A = torch.randn(L, R, K, device=dev, generator=g).bfloat16()
    B = torch.zeros(L, N, R, dtype=torch.bfloat16, device=dev)
    B[255] = torch.randn(N, R, device=dev, generator=g).bfloat16()
    x = torch.randn(M, K, device=dev, generator=g)
    adapter = torch.full((M,), -1, dtype=torch.int32, device=dev)
    adapter[0], adapter[255], adapter[100] = 255, 255, 17
    base = torch.randn(N, device=dev, generator=g).expand(M, N).contiguous()
    Y = torch.full((M, N), -7.0, device=dev)
    ws = torch.zeros(dg.dg_lora_workspace_bytes(M, K, R), dtype=torch.uint8, device=dev)
    dg.dg_lora_rows(x, A, B, adapter, Y, base=base, ws=ws)
    torch.cuda.synchronize()
    A64, B64 = A[255].double(), B[255].double()
    for m in range(M):
        if m not in (0, 255):
            assert torch.equal(Y[m], base[m]), m       # none, and one whose B is zeros
            continue
        h, ha = A64 @ x[m].double(), A64.abs() @ x[m].double().abs()
        want, mag = base[m].double() + B64 @ h, B64.abs() @ (h.abs() + (K + 1) * 2.0 ** -24 * ha)
        tol = (K + 1) * 2.0 ** -24 * (B64.abs() @ ha) + (R + 2) * 2.0 ** -24 * mag + 2.0 ** -24 * want.abs()
        assert ((Y[m].double() - want).abs() <= 1.01 * tol).all(), m


def experts_bytes(dg, dev, E, rows, cols, part):
    """Tiled Q8_0 bytes of E * rows rows of cols, which repeat `part` rows of 256 columns.  Every tile's group is laid out
    alike, so they are weights of any shape of that size."""
    import torch
    g = torch.Generator(device=dev).manual_seed(4)
    w = torch.empty(part * 8 * 34, dtype=torch.uint8, device=dev)
    dg.dg_quantize_q8_0(torch.randn(part, 256, device=dev, generator=g) / 16, w, part, 256)
    t = torch.empty(dg.dg_q8_0_tiles_bytes(part, 256), dtype=torch.uint8, device=dev)
    dg.dg_repack_q8_0_tiles(w, t, part, 256)
    return t.view(1, -1).expand(E * rows * cols // (part * 256), -1).reshape(-1)


def columns(dg, dev, M, K):
    import torch
    x = torch.randn(M, K, device=dev, generator=torch.Generator(device=dev).manual_seed(5))
    X = torch.empty(M, K // 32 * 36, dtype=torch.uint8, device=dev)
    return dg.dg_quantize_q8_1(x, X, M, K)


def test_experts_down_products(dg, dev):
    """2^26 outputs, 2^20 workgroups, of each of three experts: a token's are those that it has alone, in one launch."""
    import torch
    E, N, K, part = 3, 256, 1 << 26, 1 << 16
    W = experts_bytes(dg, dev, E, N, K, part)
    X, w = columns(dg, dev, E, K).view(E, -1), torch.tensor([[0.5], [1.0], [-2.0]], device=dev)
    ids = torch.arange(E, dtype=torch.int32, device=dev).view(E, 1)
    ws = torch.zeros(dg.dg_moe_workspace_bytes(N, K, E, 1), dtype=torch.uint8, device=dev)
    Y, alone = (torch.full((E, K), -7.0, device=dev) for _ in range(2))
    dg.dg_moe_q8_0(W, W, W, X, ids, w, Y, N, K, E, E, ws=ws)
    for m in range(E):
        dg.dg_moe_q8_0(W, W, W, X[m], ids[m:m + 1], w[m:m + 1], alone[m], N, K, 1, E, ws=ws)
    torch.cuda.synchronize()
    assert Y.isfinite().all() and (Y.abs().mean(1) > 0).all() and torch.equal(Y, alone)
    assert torch.equal(Y[:, :part], Y[:, -part:])      # the same rows


def test_experts_gated_products(dg, dev):
    """2^26 hidden values, 2^21 workgroups, of each of two experts: their columns repeat those of the rows that repeat."""
    import torch
    E, N, K, part = 2, 1 << 26, 256, 1 << 16
    W = experts_bytes(dg, dev, E, N, K, part)
    X, w = columns(dg, dev, E, K), torch.ones(E, 1, device=dev)
    ids = torch.arange(E, dtype=torch.int32, device=dev).view(E, 1)

    def hidden(n, M):
        ws = torch.zeros(dg.dg_moe_workspace_bytes(n, K, M, 1), dtype=torch.uint8, device=dev)
        Y = torch.zeros(M, K, device=dev)
        dg.dg_moe_q8_0(W, W, W, X, ids, w, Y, n, K, M, E, ws=ws)
        torch.cuda.synchronize()
        return ws[:M * (n // 32) * 36].view(M, -1)
    H, few = hidden(N, E), hidden(part, E)
    assert few.any() and torch.equal(H.view(E, N // part, -1), few.view(E, 1, -1).expand(-1, N // part, -1))
