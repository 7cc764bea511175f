"""Workloads of a decode batch in which every row has something of its own: the experts that its tokens are routed to,
the low-rank adapter of its request, the penalties, biases and grammar mask of its logits.

listed() names the measured cases, draw() makes others of the same ranges, prepare() makes one case's inputs on the
GPU, run() is one call, in plain torch (own = False) or through the library (own = True); exact() is the result in 64
bits and work() the bytes and operations a call needs.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK_BYTES = {"q4_0": 18, "q8_0": 34}


def listed():
    return [
        # the router of one token: the smallest call, all latency
        {"name": "route_f32_1x64_k6", "op": "route", "M": 1, "E": 64, "ld": 64, "k": 6, "dtype": "f32",
         "score": "softmax", "renorm": True, "scale": 1.0},
        # a prompt's tokens through a sigmoid router with a balancing bias
        {"name": "route_bf16_4096x256_k8", "op": "route", "M": 4096, "E": 256, "ld": 256, "k": 8, "dtype": "bf16",
         "score": "sigmoid", "renorm": True, "scale": 2.5},
        # one token through two of eight large 4-bit experts: bandwidth
        {"name": "moe_q4_0_8x14336x4096_k2_m1", "op": "moe", "fmt": "q4_0", "E": 8, "k": 2, "N": 14336, "K": 4096,
         "M": 1, "act": "silu", "out": "bf16", "pad": 0},
        # one token through eight of many small 4-bit experts: latency
        {"name": "moe_q4_0_128x768x2048_k8_m1", "op": "moe", "fmt": "q4_0", "E": 128, "k": 8, "N": 768, "K": 2048,
         "M": 1, "act": "silu", "out": "bf16", "pad": 0},
        # a batch with padded rows over small experts, two or three tokens to each
        {"name": "moe_q4_0_64x1536x2048_k6_m24", "op": "moe", "fmt": "q4_0", "E": 64, "k": 6, "N": 1536, "K": 2048,
         "M": 24, "act": "gelu_tanh", "out": "f16", "pad": 3},
        # the largest: a batch that reaches all of eight large 8-bit experts
        {"name": "moe_q8_0_8x14336x4096_k2_m32", "op": "moe", "fmt": "q8_0", "E": 8, "k": 2, "N": 14336, "K": 4096,
         "M": 32, "act": "silu", "out": "bf16", "pad": 0},
        # one request with an adapter beside a square projection: all latency
        {"name": "lora_bf16_1x4096x4096_r16", "op": "lora", "M": 1, "N": 4096, "K": 4096, "ld": 4096, "R": 16, "L": 4,
         "x": "bf16", "dtype": "bf16", "ranks": False, "none": 0.0},
        # a decode batch, eight adapters of several ranks, some requests without one
        {"name": "lora_f32_24x14336x4096_r64", "op": "lora", "M": 24, "N": 14336, "K": 4096, "ld": 4104, "R": 64,
         "L": 8, "x": "f32", "dtype": "f16", "ranks": True, "none": 0.2},
        # many requests, many adapters, a wide projection with an odd number of rows
        {"name": "lora_bf16_200x28669x8192_r32", "op": "lora", "M": 200, "N": 28669, "K": 8192, "ld": 8192, "R": 32,
         "L": 64, "x": "bf16", "dtype": "bf16", "ranks": False, "none": 0.1},
        # one request's logits after a short conversation
        {"name": "adjust_f32_1x128256_t600", "op": "adjust", "R": 1, "C": 128256, "ld": 128256, "dtype": "f32",
         "T": 600, "B": 16, "mask": False},
        # a serving batch with long histories, every request with penalties, some biases
        {"name": "adjust_bf16_64x128256_t8192", "op": "adjust", "R": 64, "C": 128256, "ld": 128256, "dtype": "bf16",
         "T": 8192, "B": 32, "mask": False},
        # many requests under a grammar, a vocabulary of odd length and stride
        {"name": "adjust_f16_200x32003_mask", "op": "adjust", "R": 200, "C": 32003, "ld": 32011, "dtype": "f16",
         "T": 1000, "B": 8, "mask": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "adjust"])
    if op == "route":
        E = _log_int(rng, 5, 512)
        return {"op": "route", "M": min(_log_int(rng, 1, 4096), 4096 * 256 // E), "E": E, "ld": E + rng.choice([0, 0, 3]),
                "k": min(E, rng.randint(1, 10)), "dtype": rng.choice(["f32", "f16", "bf16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5])}
    if op == "moe":
        E, K = _log_int(rng, 4, 128), 256 * _log_int(rng, 2, 28)
        N = 256 * _log_int(rng, 1, 56)
        N = max(256, min(N, 8 * 14336 * 4096 // (E * K) // 256 * 256))
        k = min(E, rng.randint(1, 8))
        M = max(1, min(_log_int(rng, 1, 48), 32 * 2 * 14336 * 4096 // (k * N * K)))
        return {"op": "moe", "fmt": rng.choice(["q4_0", "q8_0"]), "E": E, "k": k, "N": N, "K": K, "M": M,
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), "out": rng.choice(["f16", "bf16"]),
                "pad": rng.choice([0, 0, M // 4])}
    if op == "lora":
        R, K, N = rng.choice([8, 16, 32, 64, 128]), 8 * _log_int(rng, 64, 1792), _log_int(rng, 500, 28672)
        M = max(1, min(_log_int(rng, 1, 256), 200 * 32 * (28669 + 8192) // (R * (N + K))))
        L = max(1, min(_log_int(rng, 1, 64), 64 * 32 * (28669 + 8192) // (R * (N + K))))
        return {"op": "lora", "M": M, "N": N, "K": K, "ld": K + rng.choice([0, 0, 8]), "R": R, "L": L,
                "x": rng.choice(["f32", "f16", "bf16"]), "dtype": rng.choice(["f16", "bf16"]),
                "ranks": rng.random() < 0.5, "none": rng.choice([0.0, 0.3])}
    C = _log_int(rng, 1000, 150000)
    R = max(1, min(_log_int(rng, 1, 256), 64 * 128256 // C))
    T = _log_int(rng, 1, 8192)
    return {"op": "adjust", "R": R, "C": C, "ld": C + rng.choice([0, 0, 8, 5]), "dtype": rng.choice(["f32", "f16", "bf16"]),
            "T": T, "B": rng.choice([0, 4, 40]), "mask": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "route":
        M, E, k = case["M"], case["E"], case["k"]
        return {"bytes": M * E * SIZE[case["dtype"]] + (E * 4 if case["score"] == "sigmoid" else 0) + M * k * 8,
                "flops": M * E * 4}
    if op == "moe":
        E, k, N, K, M = (case[n] for n in ("E", "k", "N", "K", "M"))
        live = M - case["pad"]
        experts = E * (1 - (1 - k / E) ** live)      # distinct experts of `live` tokens, on the mean
        return {"bytes": 3 * experts * N * (K // 32) * BLOCK_BYTES[case["fmt"]] + live * (K // 32) * 36 + M * k * 8
                + 2 * M * K, "flops": 6 * live * k * N * K}
    if op == "lora":
        M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
        live = M * (1 - case["none"])
        adapters = L * (1 - (1 - 1 / L) ** live)
        share = 0.625 if case["ranks"] else 1.0      # of the rank, on the mean
        return {"bytes": adapters * R * share * (N + K) * 2 + M * K * SIZE[case["x"]] + 8 * M * N,
                "flops": 2 * live * R * share * (N + K)}
    R, C = case["R"], case["C"]
    return {"bytes": 2 * R * C * SIZE[case["dtype"]] + 4 * R * (0.75 * case["T"] + case["B"])
            + (R * C / 8 if case["mask"] else 0), "flops": R * C}


# ---- inputs ------------------------------------------------------------------------------------

def _tiles(g, fmt, rows, K):
    """Tiled bytes of a matrix of normal weights, made in that layout (a tile's order does not matter to random ones)."""
    groups = rows // 16 * (K // 256)
    dev = "cuda"
    if fmt == "q4_0":
        q = torch.randn(groups, 2, 2048, device=dev, generator=g, dtype=torch.float16).mul_(2.5).round_().clamp_(-8, 7)
        q = q.to(torch.int8).view(torch.uint8)
        codes = (q[:, 0] & 15) | (q[:, 1] << 4)
    else:
        q = torch.randn(groups, 4096, device=dev, generator=g, dtype=torch.float16).mul_(40.0).round_().clamp_(-127, 127)
        codes = q.to(torch.int8).view(torch.uint8)
    spread = 2.5 if fmt == "q4_0" else 40.0
    d = ((torch.rand(groups, 128, device=dev, generator=g) + 0.5) / (spread * math.sqrt(K))).half()
    return torch.cat([codes, d.view(torch.uint8)], 1).reshape(-1)


def _columns(g, M, K):
    """Q8_1 columns: 36-byte blocks of binary16 d, binary16 d * sum(q), 32 int8 codes."""
    q = torch.randn(M, K // 32, 32, device="cuda", generator=g).mul_(40.0).round_().clamp_(-127, 127)
    d = ((torch.rand(M, K // 32, 1, device="cuda", generator=g) + 0.5) * 0.025).half()
    s = (d.float() * q.sum(-1, keepdim=True)).half()
    return torch.cat([d.view(torch.uint8), s.view(torch.uint8), q.to(torch.int8).view(torch.uint8)], -1).reshape(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6007 + 29)
    dev = "cuda"
    st = {"case": case}
    if case["op"] == "route":
        M, E = case["M"], case["E"]
        st["x"] = (torch.randn(M, case["ld"], device=dev, generator=g) * 1.5).to(DTYPES[case["dtype"]])
        st["bias"] = torch.randn(E, device=dev, generator=g) * 0.1 if case["score"] == "sigmoid" else None
        st["ids"] = torch.zeros(M, case["k"], device=dev, dtype=torch.int32)
        st["w"] = torch.zeros(M, case["k"], device=dev)
        return st
    if case["op"] == "moe":
        E, k, N, K, M = (case[n] for n in ("E", "k", "N", "K", "M"))
        st["Wg"], st["Wu"] = (_tiles(g, case["fmt"], E * N, K) for _ in range(2))
        st["Wd"] = _tiles(g, case["fmt"], E * K, N)
        st["X"] = _columns(g, M, K)
        # what a router gives: distinct experts, weights that sum to one; rows that only fill the batch have none
        p, ids = torch.softmax(torch.randn(M, E, device=dev, generator=g) * 1.5, 1).topk(k, dim=1)
        st["w"] = p / p.sum(1, keepdim=True)
        st["ids"] = ids.to(torch.int32)
        if case["pad"]:
            st["ids"][M - case["pad"]:] = -1
        st["Y"] = torch.zeros(M, K, device=dev, dtype=DTYPES[case["out"]])
        # a program's workspace for its layers: hidden columns, the experts' sums, some room
        st["ws"] = torch.zeros(M * k * (N // 32 * 36 + 16 * K) + (4 << 20), device=dev, dtype=torch.uint8)
        return st
    if case["op"] == "lora":
        M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
        dt = DTYPES[case["dtype"]]
        st["x"] = torch.randn(M, case["ld"], device=dev, generator=g).to(DTYPES[case["x"]])
        st["A"] = (torch.randn(L, R, K, device=dev, generator=g) / math.sqrt(K)).to(dt)
        st["B"] = (torch.randn(L, N, R, device=dev, generator=g) / math.sqrt(R)).to(dt)
        a = torch.randint(0, L, (M,), device=dev, generator=g)
        st["adapter"] = torch.where(torch.rand(M, device=dev, generator=g) < case["none"], -1, a).to(torch.int32)
        st["scale"] = torch.rand(L, device=dev, generator=g) * 1.5 + 0.5
        st["ranks"] = None
        if case["ranks"]:     # eighths of the largest rank, from a quarter of it on
            st["ranks"] = (torch.randint(2, 9, (L,), device=dev, generator=g) * R // 8).to(torch.int32)
        st["base"] = torch.randn(M, N, device=dev, generator=g)
        st["Y"] = torch.zeros(M, N, device=dev)
        st["ws"] = torch.zeros(M * R * 64 + (1 << 20), device=dev, dtype=torch.uint8)
        return st
    R, C, ld, T, B = (case[n] for n in ("R", "C", "ld", "T", "B"))
    dt = DTYPES[case["dtype"]]
    st["x"] = (torch.randn(R, ld, device=dev, generator=g) * 2.5 + 1.0).to(dt)
    st["y"] = torch.zeros(R, C, device=dev, dtype=dt)
    # histories: a few tokens very often, as in text, lengths from half to the whole of T, a third of each the prompt
    r = torch.rand(R, T, device=dev, generator=g)
    st["tokens"] = (C ** (r * 0.999)).long().clamp_(0, C - 1).to(torch.int32)
    st["lens"] = (T - (torch.rand(R, device=dev, generator=g) * 0.5 * T).long()).to(torch.int32)
    st["prompt"] = st["lens"] // 3
    st["rep"] = torch.rand(R, device=dev, generator=g) * 0.4 + 1.0
    st["freq"] = torch.rand(R, device=dev, generator=g) * 0.5
    st["pres"] = torch.rand(R, device=dev, generator=g) * 0.5
    st["bias_ids"] = st["bias"] = st["mask"] = None
    if B:                 # distinct tokens of a row; one in four is forbidden
        at = (torch.arange(B, device=dev) * (C // B) + torch.randint(0, C // B, (R, B), device=dev, generator=g))
        st["bias_ids"] = at.to(torch.int32)
        v = torch.randn(R, B, device=dev, generator=g) * 4
        st["bias"] = torch.where(torch.rand(R, B, device=dev, generator=g) < 0.25, -math.inf, v)
    if case["mask"]:      # a grammar allows little at most places
        words = torch.randint(-2 ** 31, 2 ** 31, (3, R, -(-C // 32)), device=dev, generator=g)
        st["mask"] = (words[0] & words[1] & words[2]).to(torch.int32)
    return st


# ---- one call ----------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "moe": _plain_moe, "lora": _plain_lora, "adjust": _plain_adjust}[state["case"]["op"]](state)


def _run_own(st):
    import memory_bound_decode_gemv_amd as dg
    c = st["case"]
    if c["op"] == "route":
        dg.dg_moe_route(st["x"], st["ids"], st["w"], bias=st["bias"], M=c["M"], E=c["E"], ld=c["ld"], k=c["k"],
                        score=c["score"], renorm=c["renorm"], scale=c["scale"])
        return st["ids"], st["w"]
    if c["op"] == "moe":
        call = dg.dg_moe_q4_0 if c["fmt"] == "q4_0" else dg.dg_moe_q8_0
        return call(st["Wg"], st["Wu"], st["Wd"], st["X"], st["ids"], st["w"], st["Y"], N=c["N"], K=c["K"], M=c["M"],
                    E=c["E"], k=c["k"], act=c["act"], ws=st["ws"])
    if c["op"] == "lora":
        return dg.dg_lora_rows(st["x"], st["A"], st["B"], st["adapter"], st["Y"], base=st["base"], scale=st["scale"],
                               ranks=st["ranks"], M=c["M"], N=c["N"], K=c["K"], R=c["R"], L=c["L"], ld=c["ld"],
                               ws=st["ws"])
    return dg.dg_adjust_rows(st["x"], st["y"], tokens=st["tokens"], lens=st["lens"], prompt_lens=st["prompt"],
                             repetition=st["rep"], frequency=st["freq"], presence=st["pres"], bias_ids=st["bias_ids"],
                             bias=st["bias"], mask=st["mask"], R=c["R"], C=c["C"], ld=c["ld"], ldy=c["C"])


def _plain_route(st):
    c = st["case"]
    x = st["x"][:, :c["E"]].double()      # 64 bits: experts are chosen next to borders
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
    else:
        s = 1 / (1 + torch.exp(-x))
        order = torch.sort(s + st["bias"].double(), dim=1, descending=True, stable=True).indices
    ids = order[:, :c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_matrices(W, fmt, E, e, rows, K):
    """The float32 weights [len(e)][rows][K] of the experts e, from E tiled matrices."""
    T, S = rows // 16, K // 256
    b = W.view(E, T, S, 128 * BLOCK_BYTES[fmt])[e]
    n = b.shape[0]
    d = b[..., -256:].contiguous().view(torch.float16).view(n, T, S, 16, 8).permute(0, 1, 3, 2, 4).float()
    if fmt == "q4_0":
        v = b[..., :-256].reshape(n, T, S, 2, 4, 16, 4, 4).permute(0, 1, 5, 2, 3, 6, 4, 7).reshape(n, T, 16, S, 8, 16)
        q = (torch.cat([v & 15, v >> 4], -1) ^ 8).float() - 8
    else:
        v = b[..., :-256].reshape(n, T, S, 4, 4, 16, 2, 2, 4).permute(0, 1, 5, 2, 3, 6, 7, 4, 8)
        q = v.reshape(n, T, 16, S, 8, 32).view(torch.int8).float()
    return (q * d.unsqueeze(-1)).view(n, rows, K)


def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.where(g > 0, g, 0.0)


def _plain_moe(st):
    c = st["case"]
    E, k, N, K, M, fmt = (c[n] for n in ("E", "k", "N", "K", "M", "fmt"))
    b = st["X"].view(M, K // 32, 36)
    x = (b[..., 4:].view(torch.int8).float() * b[..., :2].contiguous().view(torch.float16).float()).view(M, K)
    ids, w = st["ids"].long(), torch.where(st["ids"] >= 0, st["w"], 0.0)
    if M * k < E:        # the experts of each slot; share[l, m] = the weight of expert e[l] for token m
        e = ids.reshape(-1).clamp(min=0)
        slot = torch.arange(M * k, device=x.device)
        share = torch.where((slot // k).unsqueeze(1) == torch.arange(M, device=x.device), w.reshape(-1, 1), 0.0)
    else:                # every expert
        e = torch.arange(E, device=x.device)
        share = torch.where(ids.unsqueeze(0) == e.view(-1, 1, 1), w, 0.0).sum(2)
    g = x @ _plain_matrices(st["Wg"], fmt, E, e, N, K).transpose(1, 2)
    u = x @ _plain_matrices(st["Wu"], fmt, E, e, N, K).transpose(1, 2)
    h = (_act(c["act"], g) * u).view(-1, M, N // 32, 32)
    d = (h.abs().amax(-1, keepdim=True).double() / 127).float()
    q = (h.double() / torch.where(d == 0, 1.0, d).double()).float()
    q = (q.sign() * (q.abs() + 0.5).floor()).clamp(-127, 127)
    h = (q * d.half().float()).view(-1, M, N)
    y = h @ _plain_matrices(st["Wd"], fmt, E, e, K, N).transpose(1, 2)
    return (y * share.unsqueeze(2)).sum(0).to(DTYPES[c["out"]])


def _plain_lora(st):
    c = st["case"]
    a = st["adapter"].long()
    x = st["x"][:, :c["K"]].float()
    # the products of every adapter's rank with every row, then each row's own
    h = (x @ st["A"].float().view(-1, c["K"]).t()).view(c["M"], c["L"], c["R"])
    h = h.gather(1, a.clamp(min=0).view(-1, 1, 1).expand(-1, 1, c["R"])).squeeze(1)
    if st["ranks"] is not None:
        h = torch.where(torch.arange(c["R"], device=x.device) < st["ranks"][a.clamp(min=0)].unsqueeze(1), h, 0.0)
    h = torch.where((a >= 0).unsqueeze(1), h * st["scale"][a.clamp(min=0)].unsqueeze(1), 0.0)
    mine = torch.where((a.unsqueeze(1) == torch.arange(c["L"], device=x.device)).unsqueeze(2), h.unsqueeze(1), 0.0)
    B = st["B"].float().permute(0, 2, 1).reshape(c["L"] * c["R"], c["N"])
    return st["base"] + mine.view(c["M"], -1) @ B


def _plain_adjust(st):
    c = st["case"]
    R, C, T = c["R"], c["C"], c["T"]
    v = st["x"][:, :C].float()
    at = torch.arange(T, device=v.device)
    live = at < st["lens"].unsqueeze(1)
    out = live & (at >= st["prompt"].unsqueeze(1))
    tok = st["tokens"].long()
    zeros = torch.zeros(R, C, device=v.device)
    seen = zeros.scatter_add(1, tok, live.float()) > 0
    count = zeros.scatter_add(1, tok, out.float())
    rep = st["rep"].unsqueeze(1)
    v = torch.where(seen, torch.where(v > 0, v / rep, v * rep), v)
    v = torch.where(count > 0, v - st["freq"].unsqueeze(1) * count - st["pres"].unsqueeze(1), v)
    if c["B"]:
        v = v.scatter_add(1, st["bias_ids"].long(), st["bias"])
    if c["mask"]:
        bit = torch.arange(32, device=v.device, dtype=torch.int32)
        allowed = ((st["mask"].unsqueeze(2) >> bit) & 1).view(R, -1)[:, :C]
        v = torch.where(allowed == 1, v, -math.inf)
    return v.to(st["x"].dtype)


# ---- the same in 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "moe": _exact_moe, "lora": _exact_lora, "adjust": _exact_adjust}[case["op"]](case, st)


def _exact_route(case, st):
    x = st["x"].cpu().double().numpy()[:, : case["E"]]
    if case["score"] == "softmax":
        score = np.exp(x - x.max(1)[:, None])
        score /= score.sum(1)[:, None]
        rank = x
    else:
        score = 0.5 + 0.5 * np.tanh(0.5 * x)
        rank = 1 / (1 + np.exp(-x)) + st["bias"].cpu().double().numpy()
    ids = np.argsort(-rank, axis=1, kind="stable")[:, : case["k"]]
    w = np.take_along_axis(score, ids, 1)
    if case["renorm"]:
        w /= w.sum(1)[:, None]
    return ids.astype(np.int32), w * case["scale"]


def _exact_expert(W, fmt, e, rows, K):
    """One expert's matrix in float64, tile by tile of its bytes."""
    size, S = BLOCK_BYTES[fmt], K // 256
    each = rows * (K // 32) * size
    raw = W[e * each:(e + 1) * each].view(rows // 16, S, 128 * size)
    out = torch.empty(rows // 16, 16, S, 8, 32, dtype=torch.float64, device=W.device)
    scale = raw[:, :, -256:].contiguous().view(torch.float16).reshape(-1, S, 16, 8).double()
    for block in range(8):
        for g in range(4):
            for half in range(2):
                if fmt == "q4_0":
                    at = raw[:, :, (block // 4) * 1024: (block // 4) * 1024 + 1024].reshape(-1, S, 64, 16)
                    byte = at[:, :, 16 * g:16 * g + 16, (block % 4) * 4:(block % 4) * 4 + 4].short()
                    v = (byte // (16 if half else 1)) % 16
                    v = v - 16 * (v > 7)
                else:
                    at = raw[:, :, (block // 2) * 1024: (block // 2) * 1024 + 1024].reshape(-1, S, 64, 16)
                    lo = (block % 2) * 8 + 4 * half
                    v = at[:, :, 16 * g:16 * g + 16, lo:lo + 4].contiguous().view(torch.int8)
                out[:, :, :, block, 16 * half + 4 * g:16 * half + 4 * g + 4] = v.permute(0, 2, 1, 3)
        out[:, :, :, block] *= scale[..., block].permute(0, 2, 1).unsqueeze(-1)
    return out.view(rows, K)


def _exact_moe(case, st):
    N, K, M, k, fmt = (case[n] for n in ("N", "K", "M", "k", "fmt"))
    blk = st["X"].cpu().numpy().reshape(M, K // 32, 36)
    x = torch.from_numpy((blk[..., 4:].view(np.int8) * blk[..., :2].copy().view(np.float16).astype(np.float64))
                         .reshape(M, K)).to(st["X"].device)
    ids, w = st["ids"].cpu().numpy(), st["w"].cpu().double().numpy()
    y = np.zeros((M, K))
    for e in np.unique(ids[ids >= 0]):
        m, j = np.nonzero(ids == e)
        mine = x[torch.from_numpy(m).to(x.device)]
        g = (_exact_expert(st["Wg"], fmt, int(e), N, K) @ mine.t().contiguous()).t().cpu().numpy()
        u = (_exact_expert(st["Wu"], fmt, int(e), N, K) @ mine.t().contiguous()).t().cpu().numpy()
        if case["act"] == "silu":
            a = g * (0.5 + 0.5 * np.tanh(0.5 * g))
        elif case["act"] == "gelu":
            a = g * 0.5 * torch.special.erfc(torch.from_numpy(-g * math.sqrt(0.5))).numpy()
        elif case["act"] == "gelu_tanh":
            a = g / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        else:
            a = np.maximum(g, 0)
        h = (a * u).reshape(len(m), N // 32, 32)
        d = np.max(np.abs(h), axis=-1, keepdims=True) / 127.0
        q = np.sign(h) * np.floor(np.abs(h) / np.where(d == 0, 1.0, d) + 0.5)
        h = torch.from_numpy((q * d.astype(np.float16).astype(np.float64)).reshape(len(m), N)).to(x.device)
        part = (_exact_expert(st["Wd"], fmt, int(e), K, N) @ h.t().contiguous()).t().cpu().numpy()
        np.add.at(y, m, part * w[m, j][:, None])
    return y


def _exact_lora(case, st):
    K, R = case["K"], case["R"]
    a = st["adapter"].cpu().numpy()
    y = st["base"].double()
    for e in np.unique(a[a >= 0]):
        m = torch.from_numpy(np.nonzero(a == e)[0]).to(y.device)
        r = R if st["ranks"] is None else int(st["ranks"][e])
        A, B = st["A"][e, :r].double(), st["B"][e, :, :r].double()
        y[m] += float(st["scale"][e]) * ((st["x"][m, :K].double() @ A.t()) @ B.t())
    return y


def _exact_adjust(case, st):
    C = case["C"]
    x = st["x"].cpu().double().numpy()[:, :C].copy()
    tok, lens, prompt = (st[n].cpu().numpy() for n in ("tokens", "lens", "prompt"))
    rep, freq, pres = (st[n].cpu().double().numpy() for n in ("rep", "freq", "pres"))
    for r in range(case["R"]):
        every = np.unique(tok[r, : lens[r]])
        x[r, every] = np.where(x[r, every] > 0, x[r, every] / rep[r], x[r, every] * rep[r])
        said, count = np.unique(tok[r, prompt[r]: lens[r]], return_counts=True)
        x[r, said] -= freq[r] * count + pres[r]
    if case["B"]:
        at = st["bias_ids"].cpu().numpy()
        np.put_along_axis(x, at, np.take_along_axis(x, at, 1) + st["bias"].cpu().double().numpy(), 1)
    if case["mask"]:
        bits = np.unpackbits(st["mask"].cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :C]
        x[bits == 0] = -np.inf
    return x
