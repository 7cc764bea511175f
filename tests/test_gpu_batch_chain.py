"""The operators of a batch of different requests together, as a program runs them: norm, a projection with each
request's adapter beside it, norm, router, routed experts, norm, head, each request's penalties and mask, sampler, the
token into its history (GPU)."""
import math

import numpy as np
import pytest

from tests.test_gpu_moe import STEP, Layer, route64

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Step:
    """The feed-forward half of a layer with routed experts and the tail of a step for M requests."""

    def __init__(self, dg, dev, orc, fmt, M, E=12, k=3, D=512, F=512, V=5003, R=16, L=3, T=48, seed=0):
        import torch
        self.dg, self.M, self.D, self.F, self.V, self.E, self.k, self.fmt = dg, M, D, F, V, E, k, fmt
        self.moe = Layer(dg, dev, orc, fmt, 2000 + seed, E, F, D, M, np.zeros((M, k)))
        g = self.g = torch.Generator(device=dev).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731

        def matrix(N, K, scale=1.0):
            q = torch.empty(N * (K // 32) * 34, dtype=torch.uint8, device=dev)
            return dg.dg_quantize_q8_0(randn(N, K) * (scale / math.sqrt(K)), q, N, K)
        self.proj, self.gates, self.head = matrix(D, D), matrix(E, D, 2.0), matrix(V, D, 3.0)
        self.norms = [1 + 0.1 * randn(D) for _ in range(3)]
        self.A, self.B = (randn(L, R, D) / math.sqrt(D)).bfloat16(), randn(L, D, R).bfloat16()
        self.adapter = torch.arange(M, dtype=torch.int32, device=dev) % (L + 1) - 1
        self.scale = torch.linspace(0.3, 0.8, L, device=dev)
        self.bias = 0.1 * randn(E)
        f32, u8, i32 = dict(device=dev), dict(dtype=torch.uint8, device=dev), dict(dtype=torch.int32, device=dev)
        self.x, self.h = torch.zeros(M, D, **f32), torch.zeros(M, D, **f32)
        self.n16 = torch.zeros(M, D, dtype=torch.bfloat16, device=dev)
        self.x8 = torch.zeros(M * D // 32 * 36, **u8)
        self.a, self.rl, self.y, self.logits = (torch.zeros(M, n, **f32) for n in (D, E, D, V))
        self.ids, self.w = torch.zeros(M, k, **i32), torch.zeros(M, k, **f32)
        self.idx = torch.zeros(M, dtype=torch.int64, device=dev)
        self.tokens, self.lens = torch.zeros(M, T, **i32), torch.zeros(M, **i32)
        self.prompt = torch.zeros(M, **i32)
        self.rep, self.freq, self.pres = (torch.full((M,), v, **f32) for v in (1.2, 0.3, 0.1))
        self.mask = torch.zeros(M, -(-V // 32), **i32)
        self.u, self.temp = torch.zeros(M, **f32), torch.full((M,), 0.7, **f32)
        self.top = torch.full((M,), 30, **i32)
        self.mws = torch.zeros(dg.dg_moe_workspace_bytes(F, D, M, k), **u8)
        self.lws = torch.zeros(dg.dg_lora_workspace_bytes(M, D, R), **u8)
        self.sws = torch.zeros(dg.dg_sample_workspace_bytes(M, V), **u8)
        self.new_inputs()

    def new_inputs(self):
        import torch
        M, T, V, dev = self.M, self.tokens.shape[1], self.V, self.x.device
        draw = lambda lo, hi, *s: torch.randint(lo, hi, s, device=dev, generator=self.g, dtype=torch.int32)  # noqa: E731
        self.x.copy_(torch.randn(M, self.D, device=dev, generator=self.g))
        self.h.copy_(torch.randn(M, self.D, device=dev, generator=self.g))
        self.u.copy_(torch.rand(M, device=dev, generator=self.g))
        self.tokens.copy_(draw(0, V, M, T))
        self.lens.copy_(draw(1, T - 1, M))
        self.prompt.copy_(self.lens // 2)
        self.mask.copy_(draw(-2 ** 31, 2 ** 31 - 1, *self.mask.shape))

    def state(self):
        return [t.clone() for t in (self.h, self.tokens, self.lens)]

    def set_state(self, s):
        for t, v in zip((self.h, self.tokens, self.lens), s):
            t.copy_(v)

    def run(self, keep=None):
        dg, M, D, F, V, E = self.dg, self.M, self.D, self.F, self.V, self.E
        note = (lambda **kw: None) if keep is None else (lambda **kw: keep.update({n: t.cpu() for n, t in kw.items()}))
        dg.dg_rmsnorm(self.x, self.norms[0], self.n16, res=self.h, eps=EPS)
        dg.dg_rmsnorm_q8_1(self.x, self.norms[0], self.x8, res=self.h, h=self.h, eps=EPS)
        dg.dg_gemv_q8_0(self.proj, self.x8, self.a, D, D, M)
        note(base=self.a, n16=self.n16)
        dg.dg_lora_rows(self.n16, self.A, self.B, self.adapter, self.a, base=self.a, scale=self.scale, ws=self.lws)
        dg.dg_rmsnorm_q8_1(self.a, self.norms[1], self.x8, res=self.h, h=self.h, eps=EPS)
        note(a=self.a, x8=self.x8)
        dg.dg_gemv_q8_0(self.gates, self.x8, self.rl, E, D, M)
        dg.dg_moe_route(self.rl, self.ids, self.w, bias=self.bias, score="sigmoid", scale=1.5)
        getattr(dg, f"dg_moe_{self.fmt}")(*(self.moe.tiles[n] for n in ("Wg", "Wu", "Wd")), self.x8, self.ids, self.w, self.y, F,
                                          D, M, E, ws=self.mws)
        dg.dg_rmsnorm_q8_1(self.y, self.norms[2], self.x8, res=self.h, h=self.h, eps=EPS)
        dg.dg_gemv_q8_0(self.head, self.x8, self.logits, V, D, M)
        note(logits=self.logits, tokens=self.tokens, lens=self.lens)
        dg.dg_adjust_rows(self.logits, self.logits, tokens=self.tokens, lens=self.lens, prompt_lens=self.prompt,
                          repetition=self.rep, frequency=self.freq, presence=self.pres, mask=self.mask)
        dg.dg_sample_rows(self.logits, self.u, self.idx, temperature=self.temp, top_k=self.top, ws=self.sws)
        self.tokens.scatter_(1, self.lens.long().view(M, 1), self.idx.int().view(M, 1))
        self.lens.add_(1)

    def outputs(self):
        return [t.clone() for t in (self.h, self.n16, self.x8, self.a, self.rl, self.ids, self.w, self.y, self.logits, self.idx,
                                    self.tokens, self.lens)]


@pytest.mark.parametrize("fmt,M", [("q4_0", 1), ("q8_0", 3), ("q4_0", 21)])
def test_each_link_matches_its_definition(dg, dev, orc, fmt, M):
    import torch
    from tests import test_gpu_adjust, test_gpu_sample
    s, kept = Step(dg, dev, orc, fmt, M, seed=M), {}
    s.run(kept)
    torch.cuda.synchronize()
    # the adapters' products on the projection, in place
    x, A, B = kept["n16"].double(), s.A.cpu().double(), s.B.cpu().double()
    for m, ad in enumerate(s.adapter.tolist()):
        want, tol = kept["base"][m].double(), 0.0
        if ad >= 0:
            h, dh = A[ad] @ x[m], (s.D + 1) * STEP * (A[ad].abs() @ x[m].abs())
            sc, R = float(s.scale[ad]), A.shape[1]
            want = want + sc * (B[ad] @ h)
            tol = sc * (B[ad].abs() @ dh + (R + 2) * STEP * (B[ad].abs() @ (h.abs() + dh)))
        assert ((kept["a"][m].double() - want).abs() <= 1.01 * (tol + STEP * want.abs())).all()
    # the choice, the experts
    ids, w = route64(s.rl.cpu().numpy(), s.k, "sigmoid", s.bias.cpu().numpy(), True, 1.5)
    assert np.array_equal(s.ids.cpu().numpy(), ids)
    assert (np.abs(s.w.cpu().numpy() - w) <= STEP * (1 + 2.0 ** -20) * np.abs(w)).all()
    s.moe.ids, s.moe.w, s.moe.Xq = ids, s.w.cpu().numpy(), kept["x8"].numpy().reshape(M, -1)
    H = s.mws[:M * s.k * (s.F // 32) * 36].cpu().numpy().reshape(M, s.k, -1)
    s.moe.check_hidden(H)
    s.moe.check_output(s.y.cpu().numpy(), H)
    # the tail
    a = dict(tokens=kept["tokens"].numpy(), lens=kept["lens"].numpy(), prompt_lens=s.prompt.cpu().numpy(),
             repetition=s.rep.cpu().numpy(), frequency=s.freq.cpu().numpy(), presence=s.pres.cpu().numpy(),
             mask=s.mask.cpu().numpy())
    want = torch.from_numpy(test_gpu_adjust.reference(kept["logits"].numpy(), s.V, a))
    test_gpu_adjust.same(s.logits.cpu(), want, "f32")
    for m in range(M):
        tok = test_gpu_sample.reference_row(want[m].double().numpy().copy(), float(s.u[m]), T=float(np.float32(0.7)), k=30)
        assert int(s.idx[m]) == tok == int(s.tokens[m, int(kept["lens"][m])])


@pytest.mark.parametrize("fmt,M", [("q4_0", 1), ("q8_0", 7), ("q4_0", 24)])
def test_captured_step_replays(dg, dev, orc, fmt, M):
    """Every replay, with eager work between, equals the eager step bit for bit."""
    import torch
    s = Step(dg, dev, orc, fmt, M, seed=50 + M)
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
        start = s.state()
        for t in (s.mws, s.lws):
            t.fill_(0x77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.set_state(start)
        for t in (s.x8, s.a, s.rl, s.ids, s.w, s.y, s.logits, s.idx):
            t.zero_()
        s.run()
        torch.cuda.synchronize()
        for a, b in zip(got, s.outputs()):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces(dg, dev, orc):
    import torch
    steps = [Step(dg, dev, orc, "q4_0", 9, seed=1), Step(dg, dev, orc, "q8_0", 24, E=5, k=2, seed=2)]
    want = []
    for s in steps:
        s.start = s.state()
        s.run()
        torch.cuda.synchronize()
        want.append(s.outputs())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s.set_state(s.start)
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for a, b in zip(s.outputs(), w):
                assert torch.equal(a, b)


def test_calls_one_after_another_share_a_workspace(dg, dev, orc):
    """Two layers on one stream through the same memory, eager and as two captured graphs in turn: each call is done with it
    when the next begins."""
    import torch
    s, t = Step(dg, dev, orc, "q4_0", 12, seed=5), Step(dg, dev, orc, "q8_0", 12, seed=6)
    want = []
    for c in (s, t):
        start = c.state()
        c.run()
        torch.cuda.synchronize()
        want.append(c.outputs())
        c.set_state(start)
    need = max(c.mws.numel() for c in (s, t))
    s.mws = t.mws = s.lws = t.lws = torch.full((need,), 0x11, dtype=torch.uint8, device=dev)
    starts = [c.state() for c in (s, t)]
    for c in (s, t):
        c.run()
    torch.cuda.synchronize()
    for c, w in zip((s, t), want):
        for a, b in zip(c.outputs(), w):
            assert torch.equal(a, b)
    graphs = []
    for c in (s, t):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run()
    for _ in range(3):
        for c, start in zip((s, t), starts):
            c.set_state(start)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip((s, t), want):
            for a, b in zip(c.outputs(), w):
                assert torch.equal(a, b)


def test_explicit_streams(dg, dev, orc):
    """stream= as a stream or its handle: the calls run there, behind that stream's own work."""
    import torch
    s = Step(dg, dev, orc, "q4_0", 5, seed=9)
    s.run()
    torch.cuda.synchronize()
    x8, n16, logits = s.x8.clone(), s.n16.clone(), s.logits.clone()
    side = torch.cuda.Stream()

    def calls(stream):
        y, a, z = torch.zeros_like(s.y), torch.zeros_like(s.a), torch.zeros_like(logits)
        ids, w = torch.zeros_like(s.ids), torch.zeros_like(s.w)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            late = torch.zeros_like(s.rl)
            for _ in range(50):   # work that the calls have to come after
                late.add_(s.rl / 50)
            late.copy_(s.rl)
        dg.dg_moe_route(late if stream is not None else s.rl, ids, w, stream=stream)
        dg.dg_moe_q4_0(*(s.moe.tiles[n] for n in ("Wg", "Wu", "Wd")), x8, ids, w, y, s.F, s.D, s.M, s.E, ws=s.mws, stream=stream)
        dg.dg_lora_rows(n16, s.A, s.B, s.adapter, a, base=y, scale=s.scale, ws=s.lws, stream=stream)
        dg.dg_adjust_rows(logits, z, tokens=s.tokens, lens=s.lens, repetition=s.rep, mask=s.mask, stream=stream)
        torch.cuda.synchronize()
        return [ids, w, y, a, z]
    want = calls(None)
    assert (want[0] >= 0).all()
    for stream in (side, side.cuda_stream):
        for a, b in zip(calls(stream), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_one_expert_is_the_plain_layer(dg, dev, orc, fmt):
    """A single expert with weight 1: the hidden codes are those of the gated product up to a rounding border, and the
    output is the plain tiled product of them.  (Each of the two sums is within (N/32 + 16) 2^-24 of the terms'
    magnitudes of the exact one; a code moves by less than a half with its sum's error, so by at most one.)"""
    import torch
    from tests.test_gpu_glu import columns, sums
    M, N, K = 6, 768, 512
    c = Layer(dg, dev, orc, fmt, 2100, 1, N, K, M, np.zeros((M, 1)))
    c.w[:] = 1.0
    Y, H = c.run()
    X = torch.from_numpy(c.Xq).to(dev).view(-1)
    f, y = torch.empty(M, N, device=dev), torch.empty(M, K, device=dev)
    f8 = torch.empty(M * N // 32 * 36, dtype=torch.uint8, device=dev)
    getattr(dg, f"dg_gemv_{fmt}_tiles_glu")(c.tiles["Wg"], c.tiles["Wu"], X, f, N, K, M)
    dg.dg_quantize_q8_1(f, f8, M, N)
    Hd = torch.from_numpy(H.reshape(-1)).to(dev)
    ws = torch.zeros(max(16, getattr(dg, f"dg_gemv_{fmt}_tiles_workspace_bytes")(K, N, M)), dtype=torch.uint8, device=dev)
    getattr(dg, f"dg_gemv_{fmt}_tiles")(c.tiles["Wd"], Hd, y, K, N, M, ws=ws)
    torch.cuda.synchronize()
    assert np.abs(columns(H, M, N)[1] - columns(f8.cpu().numpy(), M, N)[1]).max() <= 1
    mag = sums(fmt, c.rows["Wd"][0], H, K, N, M)[1]
    assert (np.abs(Y - y.cpu().numpy()) <= (2 * (N // 32 + 16) + 4) * STEP * mag).all()
