"""Workloads of the decode-step operators around the GEMV: residual + RMS norm into Q8_1 or
16-bit columns, the gated feed-forward product over quantised weights, and token sampling.

listed() names the measured cases, draw() makes others of the same ranges, prepare() makes one
case's inputs on the GPU, run() is one call, in plain torch (own = False) or through the library
(own = True); exact() is the result in 64 bits and work() the bytes and operations a call needs.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK_BYTES = {"q4_0": 18, "q8_0": 34}
EPS = 1e-5
WORKSPACE = 64 << 20     # bytes of device workspace that a program keeps for its calls


def listed():
    return [
        # one token of a 4096-wide model between attention and feed-forward: the smallest call, all latency
        {"name": "norm_q8_1_f32_1x4096", "op": "norm", "M": 1, "K": 4096, "ld": 4096, "dtype": "f32", "w": "f32",
         "out": "q8_1", "res": True},
        # a full decode batch of a wide model, bfloat16 residual stream
        {"name": "norm_q8_1_bf16_24x8192", "op": "norm", "M": 24, "K": 8192, "ld": 8192, "dtype": "bf16", "w": "bf16",
         "out": "q8_1", "res": True},
        # a prompt's rows into bfloat16 columns: bandwidth
        {"name": "norm_bf16_bf16_2048x8192", "op": "norm", "M": 2048, "K": 8192, "ld": 8192, "dtype": "bf16",
         "w": "f32", "out": "bf16", "res": True},
        # ragged: odd width and row stride, no residual
        {"name": "norm_f16_f16_77x2501", "op": "norm", "M": 77, "K": 2501, "ld": 2507, "dtype": "f16", "w": "f32",
         "out": "f16", "res": False},
        # one token through a decoder layer's gate and up projections, row-major Q4_0
        {"name": "glu_q4_0_14336x4096_m1", "op": "glu", "fmt": "q4_0", "tiles": False, "N": 14336, "K": 4096, "M": 1,
         "act": "silu"},
        # a ragged 8-bit matrix with a handful of columns
        {"name": "glu_q8_0_5003x2048_m5", "op": "glu", "fmt": "q8_0", "tiles": False, "N": 5003, "K": 2048, "M": 5,
         "act": "gelu_tanh"},
        # sixteen requests over the tiled copy
        {"name": "glu_q4_0_tiles_14336x4096_m16", "op": "glu", "fmt": "q4_0", "tiles": True, "N": 14336, "K": 4096,
         "M": 16, "act": "silu"},
        # the largest: a 70B-class layer in 8 bits at the most columns a call takes
        {"name": "glu_q8_0_tiles_28672x8192_m24", "op": "glu", "fmt": "q8_0", "tiles": True, "N": 28672, "K": 8192,
         "M": 24, "act": "silu"},
        # one request, one token, the usual filters
        {"name": "sample_f32_1x128256", "op": "sample", "R": 1, "C": 128256, "ld": 128256, "dtype": "f32",
         "rows": "filters", "sigma": 3.0},
        # a serving batch in which every request has filters of its own (greedy ones among them)
        {"name": "sample_bf16_64x128256_mixed", "op": "sample", "R": 64, "C": 128256, "ld": 128256, "dtype": "bf16",
         "rows": "mixed", "sigma": 2.5},
        # many requests, nearly flat distributions, top-p alone: almost the whole vocabulary stays in
        {"name": "sample_f32_256x128000_top_p", "op": "sample", "R": 256, "C": 128000, "ld": 128000, "dtype": "f32",
         "rows": "top_p", "sigma": 1.0},
        # a small vocabulary with an odd length and stride, min-p, masked tokens
        {"name": "sample_f16_5x32003", "op": "sample", "R": 5, "C": 32003, "ld": 32011, "dtype": "f16",
         "rows": "min_p", "sigma": 4.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "glu", "sample"])
    if op == "norm":
        out = rng.choice(["q8_1", "q8_1", "f32", "f16", "bf16"])
        K = 32 * _log_int(rng, 8, 512) if out == "q8_1" else _log_int(rng, 200, 16384)
        M = min(_log_int(rng, 1, 2048), 2048 * 8192 // K)
        return {"op": "norm", "M": M, "K": K, "ld": K + rng.choice([0, 0, 8, 3]),
                "dtype": rng.choice(["f32", "f16", "bf16"]), "w": rng.choice(["f32", "bf16"]), "out": out,
                "res": rng.random() < 0.7}
    if op == "glu":
        K = 256 * _log_int(rng, 2, 64)
        N = min(_log_int(rng, 500, 28672), 28672 * 8192 // K)
        return {"op": "glu", "fmt": rng.choice(["q4_0", "q8_0"]), "tiles": rng.random() < 0.5, "N": N, "K": K,
                "M": rng.randint(1, 24), "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"])}
    C = _log_int(rng, 1000, 150000)
    R = min(_log_int(rng, 1, 256), 256 * 128000 // C)
    return {"op": "sample", "R": R, "C": C, "ld": C + rng.choice([0, 0, 8, 5]),
            "dtype": rng.choice(["f32", "f16", "bf16"]), "rows": rng.choice(["filters", "mixed", "top_p", "min_p"]),
            "sigma": round(rng.uniform(0.5, 5.0), 3)}


def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        e = 4 if case["dtype"] == "f32" else 2
        o = 36 / 32 if case["out"] == "q8_1" else (4 if case["out"] == "f32" else 2)
        return {"bytes": M * K * (e * (3 if case["res"] else 1) + o) + K * (4 if case["w"] == "f32" else 2),
                "flops": 6 * M * K}
    if case["op"] == "glu":
        N, K, M = case["N"], case["K"], case["M"]
        return {"bytes": 2 * N * (K // 32) * BLOCK_BYTES[case["fmt"]] + M * (K // 32) * 36 + 4 * M * N,
                "flops": 4 * N * K * M}
    e = 4 if case["dtype"] == "f32" else 2
    return {"bytes": case["R"] * case["C"] * e + case["R"] * 28, "flops": 4 * case["R"] * case["C"]}


# ---- inputs ------------------------------------------------------------------------------------

def _weights(g, fmt, tiles, N, K):
    """One matrix's bytes: codes of normal weights and binary16 block scales, rows of blocks or 16-row tiles."""
    dev = "cuda"
    nb = K // 32
    rows = -(-N // 16) * 16 if tiles else N
    spread, zero = (2.5, 8) if fmt == "q4_0" else (40.0, 0)
    q = torch.randn(N, nb, 32, device=dev, generator=g, dtype=torch.float16).mul_(spread).round_()
    q = q.clamp_(-8, 7) if fmt == "q4_0" else q.clamp_(-127, 127)
    q = q.to(torch.int8)
    d = ((torch.rand(N, nb, device=dev, generator=g) + 0.5) * (0.025 / spread)).half()
    if rows > N:
        q = torch.cat([q, torch.zeros(rows - N, nb, 32, device=dev, dtype=torch.int8)])
        d = torch.cat([d, torch.zeros(rows - N, nb, device=dev, dtype=torch.float16)])
    if not tiles:
        if fmt == "q4_0":
            u = (q + zero).view(torch.uint8)
            codes = u[..., :16] | (u[..., 16:] << 4)
        else:
            codes = q.view(torch.uint8)
        return torch.cat([d.unsqueeze(-1).view(torch.uint8), codes], -1).reshape(-1)
    T, S = rows // 16, nb // 8
    dt = d.view(T, 16, S, 8).permute(0, 2, 1, 3).contiguous().view(torch.uint8).reshape(T, S, 256)
    if fmt == "q4_0":
        u = q.view(torch.uint8) & 15                       # two's-complement nibbles of q - 8
        c = u[..., :16] | (u[..., 16:] << 4)               # row, block, byte
        c = c.view(T, 16, S, 2, 4, 4, 4).permute(0, 2, 3, 5, 1, 4, 6)     # tile, group, half, g, n, block, byte
    else:
        c = q.view(torch.uint8).view(T, 16, S, 4, 2, 2, 4, 4).permute(0, 2, 3, 6, 1, 4, 5, 7)
    return torch.cat([c.reshape(T, S, -1), dt], -1).reshape(-1)


def _columns(g, M, K):
    """Q8_1 columns: 36-byte blocks of binary16 d, binary16 d * sum(q), 32 int8 codes."""
    q = torch.randn(M, K // 32, 32, device="cuda", generator=g).mul_(40.0).round_().clamp_(-127, 127)
    d = ((torch.rand(M, K // 32, 1, device="cuda", generator=g) + 0.5) * 0.02).half()
    s = (d.float() * q.sum(-1, keepdim=True)).half()
    return torch.cat([d.view(torch.uint8), s.view(torch.uint8), q.to(torch.int8).view(torch.uint8)], -1).reshape(-1)


def _row_parameters(rows, R, r):
    """Per-row temperature, top-k, top-p, min-p of a batch."""
    T = r.uniform(0.6, 1.3, R)
    k, p, mp = np.zeros(R), np.ones(R), np.zeros(R)
    if rows == "filters":
        k, p, mp = r.choice([20, 40, 50, 64], R), r.uniform(0.8, 0.98, R), np.full(R, 0.02)
    elif rows == "top_p":
        p = r.uniform(0.9, 0.999, R)
    elif rows == "min_p":
        mp = r.uniform(0.02, 0.1, R)
    else:
        kind = r.integers(0, 6, R)
        T = np.where(kind == 0, 0.0, T)                                  # greedy
        k = np.where((kind == 1) | (kind == 4), r.integers(1, 200, R), 0)
        p = np.where((kind == 2) | (kind == 4), r.uniform(0.5, 0.99, R), 1.0)
        mp = np.where((kind == 3) | (kind == 4), r.uniform(0.01, 0.2, R), 0.0)   # kind 5: temperature alone
    return T, k, p, mp


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    dev = "cuda"
    st = {"case": case}
    if case["op"] == "norm":
        M, K, ld = case["M"], case["K"], case["ld"]
        dt = DTYPES[case["dtype"]]
        scale = torch.rand(M, 1, device=dev, generator=g) * 3 + 0.2
        st["x"] = (torch.randn(M, ld, device=dev, generator=g) * scale).to(dt)
        st["w"] = (1 + 0.2 * torch.randn(K, device=dev, generator=g)).to(DTYPES[case["w"]])
        st["res"] = (torch.randn(M, ld, device=dev, generator=g) * 2).to(dt) if case["res"] else None
        st["h"] = torch.zeros(M, ld, device=dev, dtype=dt) if case["res"] else None
        if case["out"] == "q8_1":
            st["y"] = torch.zeros(M * (K // 32) * 36, device=dev, dtype=torch.uint8)
        else:
            st["y"] = torch.zeros(M, K, device=dev, dtype=DTYPES[case["out"]])
        return st
    st["ws"] = torch.zeros(WORKSPACE, device=dev, dtype=torch.uint8)
    if case["op"] == "glu":
        N, K, M = case["N"], case["K"], case["M"]
        st["Wg"] = _weights(g, case["fmt"], case["tiles"], N, K)
        st["Wu"] = _weights(g, case["fmt"], case["tiles"], N, K)
        st["X"] = _columns(g, M, K)
        st["Y"] = torch.zeros(M, N, device=dev)
        return st
    R, C, ld = case["R"], case["C"], case["ld"]
    x = torch.randn(R, ld, device=dev, generator=g) * case["sigma"] + 2.0
    # a few tokens that stand out, as a language model's logits have them
    top = torch.randint(0, C, (R, 8), device=dev, generator=g)
    x.scatter_add_(1, top, torch.rand(R, 8, device=dev, generator=g) * 4 * case["sigma"])
    if case["rows"] == "min_p":      # tokens that a grammar forbids
        x.masked_fill_(torch.rand(R, ld, device=dev, generator=g) < 0.3, float("-inf"))
    st["x"] = x.to(DTYPES[case["dtype"]])
    T, k, p, mp = _row_parameters(case["rows"], R, np.random.default_rng(seed))
    st["T"] = torch.tensor(T, device=dev, dtype=torch.float32)
    st["k"] = torch.tensor(k, device=dev, dtype=torch.int32)
    st["p"] = torch.tensor(p, device=dev, dtype=torch.float32)
    st["mp"] = torch.tensor(mp, device=dev, dtype=torch.float32)
    st["u"] = torch.rand(R, device=dev, generator=g)
    st["idx"] = torch.zeros(R, device=dev, dtype=torch.int64)
    return st


# ---- one call ----------------------------------------------------------------------------------

def _q8_1_values(y, M, K):
    """Codes times the block's binary16 scale, as stored."""
    b = y.view(M, K // 32, 36)
    return b[..., 4:].view(torch.int8) * b[..., :2].view(torch.float16)


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "glu": _plain_glu, "sample": _plain_sample}[state["case"]["op"]](state)


def _run_own(state):
    import memory_bound_decode_gemv_amd as dg
    c = state["case"]
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        call = dg.dg_rmsnorm_q8_1 if c["out"] == "q8_1" else dg.dg_rmsnorm
        call(state["x"], state["w"], state["y"], M=M, K=K, ld=c["ld"], res=state["res"], h=state["h"], eps=EPS)
        y = _q8_1_values(state["y"], M, K) if c["out"] == "q8_1" else state["y"]
        return (y, state["h"][:, :K]) if c["res"] else (y,)
    if c["op"] == "glu":
        name = "dg_gemv_%s%s_glu" % (c["fmt"], "_tiles" if c["tiles"] else "")
        getattr(dg, name)(state["Wg"], state["Wu"], state["X"], state["Y"], c["N"], c["K"], c["M"], act=c["act"])
        return state["Y"]
    dg.dg_sample_rows(state["x"], state["u"], state["idx"], R=c["R"], C=c["C"], ld=c["ld"], temperature=state["T"],
                      top_k=state["k"], top_p=state["p"], min_p=state["mp"], ws=state["ws"])
    return state["idx"]


def _plain_norm(state):
    c = state["case"]
    M, K = c["M"], c["K"]
    x = state["x"][:, :K]
    h = x
    if c["res"]:
        h = (x.float() + state["res"][:, :K].float()).to(x.dtype)
    hf = h.float()
    # the long sum and the root in 64 bits: the codes below sit next to rounding borders
    r = (1.0 / (hf.double().square().sum(1, keepdim=True) / K + float(np.float32(EPS))).sqrt()).float()
    y = (hf * r) * state["w"].float()
    if c["out"] != "q8_1":
        y = y.to(DTYPES[c["out"]])
        return (y, h) if c["res"] else (y,)
    b = y.view(M, K // 32, 32)
    d = (b.abs().amax(-1, keepdim=True).double() / 127).float()
    v = (b.double() / torch.where(d == 0, 1.0, d).double()).float().double()
    q = (v.sign() * (v.abs() + 0.5).floor()).clamp(-127, 127)
    y = q.to(torch.int8) * d.half()
    return (y, h) if c["res"] else (y,)


def _plain_matrix(W, fmt, tiles, N, K):
    """The float32 weights of packed bytes."""
    nb = K // 32
    if not tiles:
        b = W[: N * nb * BLOCK_BYTES[fmt]].view(N, nb, BLOCK_BYTES[fmt])
        d = b[..., :2].contiguous().view(torch.float16).float()
        c = b[..., 2:]
        q = (torch.cat([c & 15, c >> 4], -1).float() - 8) if fmt == "q4_0" else c.view(torch.int8).float()
        return (q * d).view(N, K)
    T, S = -(-N // 16), nb // 8
    b = W[: T * S * 128 * BLOCK_BYTES[fmt]].view(T, S, 128 * BLOCK_BYTES[fmt])
    d = b[..., -256:].contiguous().view(torch.float16).view(T, S, 16, 8).permute(0, 2, 1, 3).float()
    if fmt == "q4_0":
        c = b[..., :-256].reshape(T, S, 2, 4, 16, 4, 4).permute(0, 4, 1, 2, 5, 3, 6).reshape(T, 16, S, 8, 16)
        q = ((torch.cat([c & 15, c >> 4], -1) ^ 8).float() - 8)
    else:
        c = b[..., :-256].reshape(T, S, 4, 4, 16, 2, 2, 4).permute(0, 4, 1, 2, 5, 6, 3, 7)
        q = c.reshape(T, 16, S, 8, 32).view(torch.int8).float()
    return (q * d.unsqueeze(-1)).view(T * 16, K)[:N]


def _plain_glu(state):
    c = state["case"]
    N, K, M = c["N"], c["K"], c["M"]
    b = state["X"].view(M, K // 32, 36)
    x = (b[..., 4:].view(torch.int8).float() * b[..., :2].contiguous().view(torch.float16).float()).view(M, K)
    g = x @ _plain_matrix(state["Wg"], c["fmt"], c["tiles"], N, K).t()
    u = x @ _plain_matrix(state["Wu"], c["fmt"], c["tiles"], N, K).t()
    if c["act"] == "silu":
        a = g / (1 + torch.exp(-g))
    elif c["act"] == "gelu":
        a = 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    else:
        a = torch.where(g > 0, g, 0.0)
    return a * u


def _plain_sample(state):
    # 64 bits throughout: tokens are decided next to borders of long sums
    C = state["case"]["C"]
    x = state["x"][:, :C].double()
    T, p, mp = (state[n].double().unsqueeze(1) for n in ("T", "p", "mp"))
    k = state["k"].unsqueeze(1)
    at = torch.arange(C, device=x.device)
    m = x.amax(1, keepdim=True)
    greedy = torch.where(x == m, at, C).amin(1)
    w = torch.exp((x - m) / torch.where(T > 0, T, 1.0))
    w = torch.where(x == -math.inf, 0.0, w)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    keep = (at < k) | (k <= 0)
    cum = torch.cumsum(ws * keep, 1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    keep &= (before < p * cum[:, -1:]) | (p >= 1) | (at == 0)
    keep &= ws >= mp.clamp(max=1.0)
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    cum = torch.cumsum(w * kept, 1)
    total = cum[:, -1:]
    idx = (cum <= state["u"].double().unsqueeze(1) * total).sum(1)
    idx = torch.where(total.squeeze(1) > 0, idx, -1)
    return torch.where(state["T"] > 0, idx, greedy)


# ---- the same in 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "glu": _exact_glu, "sample": _exact_sample}[case["op"]](case, st)


def _exact_norm(case, st):
    K = case["K"]
    h = st["x"][:, :K].cpu().double().numpy()
    if case["res"]:
        h = h + st["res"][:, :K].cpu().double().numpy()
        h = torch.from_numpy(h).to(st["x"].dtype).double().numpy()      # what the residual stream stores
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(np.float32(EPS))) * st["w"].cpu().double().numpy()
    if case["out"] == "q8_1":
        b = y.reshape(case["M"], K // 32, 32)
        d = np.max(np.abs(b), axis=-1, keepdims=True) / 127.0
        q = np.sign(b) * np.floor(np.abs(b) / np.where(d == 0, 1.0, d) + 0.5)
        y = q * d.astype(np.float16).astype(np.float64)
    return (y, h) if case["res"] else (y,)


def _exact_rows(W, case, n0, n1):
    """Rows n0..n1 (n0 a multiple of 16) of a packed matrix, float64, on the matrix's device."""
    nb, fmt = case["K"] // 32, case["fmt"]
    size = BLOCK_BYTES[fmt]
    if not case["tiles"]:
        blk = W.reshape(-1, nb, size)[n0:n1]
        d = blk[..., :2].contiguous().view(torch.float16).double()
        q = torch.empty(n1 - n0, nb, 32, dtype=torch.float64, device=W.device)
        if fmt == "q8_0":
            q[:] = blk[..., 2:].view(torch.int8)
        else:
            q[..., :16], q[..., 16:] = blk[..., 2:] % 16, blk[..., 2:] // 16
            q -= 8
        return (q * d).reshape(n1 - n0, case["K"])
    groups = nb // 8
    t0, t1 = n0 // 16, -(-n1 // 16)
    raw = W.reshape(-1, groups, 128 * size)[t0:t1]
    out = torch.zeros(t1 - t0, 16, groups, 8, 32, dtype=torch.float64, device=W.device)
    scales = raw[:, :, -256:].contiguous().view(torch.float16).reshape(t1 - t0, groups, 16, 8).double()
    for block in range(8):
        for g in range(4):
            for row in range(16):
                lane = 16 * g + row
                to = out[:, row, :, block]
                if fmt == "q4_0":
                    at = (block // 4) * 1024 + lane * 16 + (block % 4) * 4
                    byte = raw[:, :, at:at + 4].short()
                    to[..., 4 * g:4 * g + 4] = (byte % 16 + 8) % 16 - 8
                    to[..., 16 + 4 * g:20 + 4 * g] = (byte // 16 + 8) % 16 - 8
                else:
                    at = (block // 2) * 1024 + lane * 16 + (block % 2) * 8
                    byte = raw[:, :, at:at + 8].contiguous().view(torch.int8)
                    to[..., 4 * g:4 * g + 4] = byte[..., :4]
                    to[..., 16 + 4 * g:20 + 4 * g] = byte[..., 4:]
        out[:, :, :, block] *= scales[..., block].transpose(1, 2).unsqueeze(-1)
    return out.reshape((t1 - t0) * 16, case["K"])[: n1 - n0]


def _exact_glu(case, st):
    N, K, M = case["N"], case["K"], case["M"]
    blk = st["X"].cpu().numpy().reshape(M, K // 32, 36)
    x = blk[..., 4:].view(np.int8) * blk[..., :2].copy().view(np.float16).astype(np.float64)
    x = torch.from_numpy(x.reshape(M, K)).to(st["X"].device)
    parts = []
    for n0 in range(0, N, 4096):
        n1 = min(N, n0 + 4096)
        g, u = ((x @ _exact_rows(st[name], case, n0, n1).t().contiguous()).cpu().numpy() for name in ("Wg", "Wu"))
        if case["act"] == "silu":
            a = g * (0.5 + 0.5 * np.tanh(0.5 * g))
        elif case["act"] == "gelu":
            a = g * 0.5 * torch.special.erfc(torch.from_numpy(-g * math.sqrt(0.5))).numpy()
        elif case["act"] == "gelu_tanh":
            a = g / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        else:
            a = np.maximum(g, 0)
        parts.append(a * u)
    return np.concatenate(parts, axis=1)


def _exact_sample(case, st):
    rows = st["x"][:, : case["C"]].cpu().double().numpy()
    T, k, p, mp, u = (st[n].cpu().double().numpy() for n in ("T", "k", "p", "mp", "u"))
    out = np.empty(case["R"], dtype=np.int64)
    for r, x in enumerate(rows):
        if not T[r] > 0:
            out[r] = int(np.argmax(x))
            continue
        m = x.max()
        if m == -np.inf:
            out[r] = -1
            continue
        w = np.exp((x - m) / T[r])
        rank = np.argsort(-x, kind="stable")
        if k[r] > 0:
            rank = rank[: int(k[r])]
        if p[r] < 1:
            sums = np.cumsum(w[rank], dtype=np.longdouble)
            rank = rank[: int(np.searchsorted(sums, np.longdouble(p[r]) * sums[-1])) + 1]
        kept = np.sort(rank[w[rank] >= min(mp[r], 1.0)])
        sums = np.cumsum(w[kept], dtype=np.longdouble)
        out[r] = kept[int(np.searchsorted(sums, np.longdouble(u[r]) * sums[-1], side="right"))]
    return out
