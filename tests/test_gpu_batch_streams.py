"""stream= of the operators of a batch of different requests: a call comes after its stream's own work (GPU).

Each operator reads an input that its stream makes late, behind some tens of milliseconds of products that are still
under way when every call has been issued.  A call on another stream would not wait for them and read what was there
before."""
import pytest

from tests.test_gpu_moe import Layer, distinct

pytestmark = pytest.mark.gpu


class Operators:
    """One call of each, the late input's first contents (which give other results), and its later ones."""

    def __init__(self, dg, dev, orc):
        import torch
        self.dg, self.dev = dg, dev
        g = torch.Generator(device=dev).manual_seed(77)
        randn = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
        M, E, k, N, K = 5, 12, 3, 512, 512
        self.moe = Layer(dg, dev, orc, "q4_0", 4100, E, N, K, M, distinct(1, E, M, k))
        self.shape = (N, K, M, E)
        self.x8 = torch.from_numpy(self.moe.Xq.reshape(-1)).to(dev)
        self.w = torch.full((M, k), 0.5, device=dev)
        self.A, self.B = randn(2, 16, K) / 20, randn(2, 300, 16)
        self.A, self.B = self.A.bfloat16(), self.B.bfloat16()
        self.adapter = torch.arange(M, dtype=torch.int32, device=dev) % 2
        self.tokens = torch.arange(M * 9, dtype=torch.int32, device=dev).view(M, 9)
        self.rep = torch.full((M,), 1.5, device=dev)
        ids = torch.from_numpy(self.moe.ids).to(dev)
        self.late = {"route": (randn(M, E), randn(M, E)), "moe": ((ids + 1) % E, ids), "lora": (randn(M, K), randn(M, K)),
                     "adjust": (randn(M, 5003), randn(M, 5003))}
        self.mws = torch.zeros(dg.dg_moe_workspace_bytes(N, K, M, k), dtype=torch.uint8, device=dev)
        self.lws = torch.zeros(dg.dg_lora_workspace_bytes(M, K, 16), dtype=torch.uint8, device=dev)

    def outputs(self):
        import torch
        M, dev = 5, self.dev
        return {"route": [torch.full((M, 3), -5, dtype=torch.int32, device=dev), torch.zeros(M, 3, device=dev)],
                "moe": [torch.zeros(M, 512, device=dev)], "lora": [torch.zeros(M, 300, device=dev)],
                "adjust": [torch.zeros(M, 5003, device=dev)]}

    def call(self, name, x, out, stream):
        dg, t = self.dg, self.moe.tiles
        if name == "route":
            dg.dg_moe_route(x, *out, stream=stream)
        elif name == "moe":
            dg.dg_moe_q4_0(t["Wg"], t["Wu"], t["Wd"], self.x8, x, self.w, out[0], *self.shape, ws=self.mws, stream=stream)
        elif name == "lora":
            dg.dg_lora_rows(x, self.A, self.B, self.adapter, out[0], ws=self.lws, stream=stream)
        else:
            dg.dg_adjust_rows(x, out[0], tokens=self.tokens, repetition=self.rep, stream=stream)


@pytest.mark.parametrize("handle", [False, True])
def test_each_call_waits_for_its_streams_work(dg, dev, orc, handle):
    import torch
    ops = Operators(dg, dev, orc)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    big = torch.ones(8192, 8192, dtype=torch.bfloat16, device=dev)
    product = torch.mm(big, big)
    results = {}
    for name, (before, after) in ops.late.items():
        early, want = ops.outputs()[name], ops.outputs()[name]
        ops.call(name, before, early, None)
        ops.call(name, after, want, None)
        results[name] = (early, want)
    torch.cuda.synchronize()
    for name, (early, want) in results.items():
        assert not torch.equal(early[-1], want[-1]), name
    x = {name: before.clone() for name, (before, _) in ops.late.items()}
    out = ops.outputs()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):      # some 50 ms: an 8192^3 product takes 0.9
            torch.mm(big, big, out=product)
        for name, (_, after) in ops.late.items():
            x[name].copy_(after)
    for name in ops.late:
        ops.call(name, x[name], out[name], stream)
    late = not side.query()
    torch.cuda.synchronize()
    assert late, "the products ended before the calls were issued"
    for name, (_, want) in results.items():
        for a, b in zip(out[name], want):
            assert torch.equal(a, b), name
