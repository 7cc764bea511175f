"""The decode-step operators together, as a program runs them: residual and norm into Q8_1, the gated product, the down
projection, the next norm, the head, the sampler (GPU)."""
import math

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Step:
    """Feed-forward half of a layer and the tail of a step for M requests, from quantised weights."""

    def __init__(self, dg, dev, fmt, tiles, M, D=1024, F=2304, V=9000, seed=0):
        import torch
        self.dg, self.M, self.D, self.F, self.V, self.fmt, self.tiles = dg, M, D, F, V, fmt, tiles
        g = torch.Generator(device=dev).manual_seed(seed)
        self.g = g
        block = 18 if fmt == "q4_0" else 34

        def matrix(N, K, tiled):
            w = torch.randn(N, K, device=dev, generator=g) / math.sqrt(K)
            q = torch.empty(N * (K // 32) * block, dtype=torch.uint8, device=dev)
            getattr(dg, f"dg_quantize_{fmt}")(w, q, N, K)
            if not tiled:
                return q
            t = torch.empty(getattr(dg, f"dg_{fmt}_tiles_bytes")(N, K), dtype=torch.uint8, device=dev)
            getattr(dg, f"dg_repack_{fmt}_tiles")(q, t, N, K)
            return t
        self.gate, self.up, self.down = matrix(F, D, tiles), matrix(F, D, tiles), matrix(D, F, tiles)
        self.head = matrix(V, D, False)
        self.w1 = 1 + 0.1 * torch.randn(D, device=dev, generator=g)
        self.w2 = 1 + 0.1 * torch.randn(D, device=dev, generator=g)
        f32, u8 = dict(device=dev), dict(dtype=torch.uint8, device=dev)
        self.x, self.h = torch.zeros(M, D, **f32), torch.zeros(M, D, **f32)
        self.u = torch.zeros(M, **f32)
        self.x8, self.f8 = torch.zeros(M * D // 32 * 36, **u8), torch.zeros(M * F // 32 * 36, **u8)
        self.f, self.y, self.logits = torch.zeros(M, F, **f32), torch.zeros(M, D, **f32), torch.zeros(M, V, **f32)
        self.n16 = torch.zeros(M, D, dtype=torch.bfloat16, device=dev)
        self.T, self.p = torch.full((M,), 0.8, **f32), torch.full((M,), 0.95, **f32)
        self.k = torch.full((M,), 40, dtype=torch.int32, device=dev)
        self.idx = torch.zeros(M, dtype=torch.int64, device=dev)
        need = max(getattr(dg, f"dg_gemv_{fmt}_tiles_workspace_bytes")(D, F, M), 16)
        self.ws = torch.zeros(need, **u8)
        self.sws = torch.zeros(dg.dg_sample_workspace_bytes(M, V), **u8)
        self.new_inputs()

    def new_inputs(self):
        import torch
        self.x.copy_(torch.randn(self.M, self.D, device=self.x.device, generator=self.g))
        self.h.copy_(torch.randn(self.M, self.D, device=self.x.device, generator=self.g) * 2)
        self.u.copy_(torch.rand(self.M, device=self.x.device, generator=self.g))

    def run(self):
        dg, M, D, F, V, fmt = self.dg, self.M, self.D, self.F, self.V, self.fmt
        dg.dg_rmsnorm_q8_1(self.x, self.w1, self.x8, res=self.h, h=self.h, eps=EPS)
        if self.tiles:
            getattr(dg, f"dg_gemv_{fmt}_tiles_glu")(self.gate, self.up, self.x8, self.f, F, D, M)
        else:
            getattr(dg, f"dg_gemv_{fmt}_glu")(self.gate, self.up, self.x8, self.f, F, D, M)
        dg.dg_quantize_q8_1(self.f, self.f8, M, F)
        if self.tiles:
            getattr(dg, f"dg_gemv_{fmt}_tiles")(self.down, self.f8, self.y, D, F, M, ws=self.ws)
        else:
            getattr(dg, f"dg_gemv_{fmt}")(self.down, self.f8, self.y, D, F, M)
        dg.dg_rmsnorm(self.y, self.w2, self.n16, res=self.h, eps=EPS)
        dg.dg_rmsnorm_q8_1(self.y, self.w2, self.x8, res=self.h, h=self.h, eps=EPS)
        getattr(dg, f"dg_gemv_{fmt}")(self.head, self.x8, self.logits, V, D, M)
        dg.dg_sample_rows(self.logits, self.u, self.idx, temperature=self.T, top_k=self.k, top_p=self.p, ws=self.sws)

    def outputs(self):
        return [t.clone() for t in (self.h, self.x8, self.f, self.y, self.n16, self.logits, self.idx)]


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("tiles,M", [(False, 1), (False, 3), (True, 7), (True, 20)])
def test_each_link_matches_its_definition(dg, dev, orc, fmt, tiles, M):
    import torch
    from tests import test_gpu_glu, test_gpu_norm, test_gpu_sample
    s = Step(dg, dev, fmt, tiles, M, seed=M)
    plain = Step(dg, dev, fmt, False, M, seed=M)   # the same weights, row-major
    x, h = s.x.cpu(), s.h.cpu()
    s.run()
    torch.cuda.synchronize()
    h1, y32, _ = test_gpu_norm.reference(x, h, s.w1.cpu(), EPS)
    x8 = orc.quantize_q8_1(y32)
    G, U = (test_gpu_glu.sums(fmt, w.cpu().numpy(), x8, s.F, s.D, M) for w in (plain.gate, plain.up))
    f = s.f.cpu().numpy()
    test_gpu_glu.check("silu", f, G, U, s.D)
    f8 = orc.quantize_q8_1(f)
    assert np.array_equal(s.f8.cpu().numpy(), f8.reshape(-1))
    want, mag = test_gpu_glu.sums(fmt, plain.down.cpu().numpy(), f8, s.D, s.F, M)
    y = s.y.cpu()
    assert (np.abs(y.numpy() - want) <= (s.F // 32 + 16) * 2.0 ** -24 * mag).all()
    h2, y32, _ = test_gpu_norm.reference(y, h1, s.w2.cpu(), EPS)
    assert torch.equal(s.h.cpu(), h2)
    assert torch.equal(s.n16.cpu(), torch.from_numpy(y32).bfloat16())
    x8 = orc.quantize_q8_1(y32)
    assert np.array_equal(s.x8.cpu().numpy(), x8.reshape(-1))
    logits = s.logits.cpu().double().numpy()
    for r in range(M):
        want = test_gpu_sample.reference_row(logits[r].copy(), float(s.u[r]), T=float(np.float32(0.8)), k=40,
                                             p=float(np.float32(0.95)))
        assert int(s.idx[r]) == want


@pytest.mark.parametrize("fmt,tiles,M", [("q4_0", False, 1), ("q4_0", True, 12), ("q8_0", False, 9), ("q8_0", True, 24)])
def test_captured_step_replays(dg, dev, fmt, tiles, M):
    """Every replay, with eager work between, equals the eager step bit for bit."""
    import torch
    s = Step(dg, dev, fmt, tiles, M, seed=100 + M)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(4):
        s.new_inputs()
        h = s.h.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.h.copy_(h)
        for t in (s.x8, s.f, s.f8, s.y, s.n16, s.logits, s.idx):
            t.zero_()
        s.run()
        torch.cuda.synchronize()
        for a, b in zip(got, s.outputs()):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces(dg, dev):
    import torch
    steps = [Step(dg, dev, "q4_0", True, 16, seed=1), Step(dg, dev, "q8_0", True, 24, seed=2)]
    want = []
    for s in steps:
        h = s.h.clone()
        s.run()
        torch.cuda.synchronize()
        want.append(s.outputs())
        s.h0 = h
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s.h.copy_(s.h0)
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for a, b in zip(s.outputs(), w):
                assert torch.equal(a, b)
