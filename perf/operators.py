"""Cases of the operators around the draft cycle, for timing and comparison: RMS norm (bf16 and int8 output), row
quantisation, the int8 matrix product, and log-probabilities of given or emitted tokens.

`own` false: every operator in its plain form, elementary torch operations.  `own` true: the calls a user makes of
block_draft_selection_b200.  Both take what `prepare` gives.
"""
import math

import torch

own = False

_pkg = None


def _lib():
    global _pkg
    if _pkg is None:
        import block_draft_selection_b200
        _pkg = block_draft_selection_b200
    return _pkg


# ---------------------------------------------------------------- cases ---

def listed():
    return [
        # one block of 8 positions before the LM head: what counts is latency
        {"name": "norm_i8 one block", "op": "norm", "M": 8, "d": 2560, "residual": True, "i8": True},
        # 256 blocks of 17 positions, the throughput workload's hidden size
        {"name": "norm_i8 throughput", "op": "norm", "M": 4352, "d": 4096, "residual": True, "i8": True},
        # an odd number of rows, bf16 out for the bf16 LM head, no residual
        {"name": "norm_bf16 ragged", "op": "norm", "M": 447, "d": 5120, "residual": False, "i8": False},
        # a vocabulary's head laid out in int8, once per weight set
        {"name": "quant head", "op": "quant", "M": 151936, "d": 2560},
        # hidden states of 16 blocks of 6 positions quantised at every step
        {"name": "quant step", "op": "quant", "M": 96, "d": 5120},
        # the int8 head at batch 1: weight streaming
        {"name": "gemm head one block", "op": "gemm", "M": 8, "N": 151936, "K": 2560, "bf16": False},
        # the int8 head of 16 blocks of 6 positions, bf16 logits
        {"name": "gemm head 16 blocks", "op": "gemm", "M": 96, "N": 151936, "K": 5120, "bf16": True},
        # a projection of a batch, odd in both outer sizes
        {"name": "gemm projection odd", "op": "gemm", "M": 333, "N": 4099, "K": 2576, "bf16": False},
        # the int8 head of the throughput workload: tensor bound
        {"name": "gemm head throughput", "op": "gemm", "M": 4352, "N": 129280, "K": 4096, "bf16": False},
        # one step's 8 rows of logits: latency
        {"name": "logprobs one block", "op": "logprobs", "M": 8, "V": 151936, "pad": 0, "bf16": False, "K": 16,
         "T": 1.0, "masked": 0.0},
        # a prompt's rows of bf16 logits in a padded, strided buffer, vocabulary masked in part
        {"name": "logprobs prompt bf16", "op": "logprobs", "M": 513, "V": 151643, "pad": 293, "bf16": True, "K": 20,
         "T": 0.7, "masked": 0.3},
        # tokens emitted by a verification step of 256 blocks of 16 drafts
        {"name": "emitted throughput", "op": "emitted", "B": 256, "L": 16, "V": 129280, "K": 16, "T": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "gemm", "gemm", "gemm", "logprobs", "logprobs", "emitted"])
    if op == "norm":
        return {"op": op, "M": _log_int(rng, 1, 4352), "d": 8 * _log_int(rng, 1, 1024),
                "residual": rng.random() < 0.7, "i8": rng.random() < 0.6}
    if op == "quant":
        d = 8 * _log_int(rng, 1, 1024)
        return {"op": op, "M": _log_int(rng, 1, min(151936, 151936 * 2560 // d)), "d": d}
    if op == "gemm":
        while True:
            c = {"op": op, "M": _log_int(rng, 1, 4352), "N": _log_int(rng, 1, 151936), "K": 16 * _log_int(rng, 1, 320),
                 "bf16": rng.random() < 0.4}
            if c["M"] * c["N"] <= 4352 * 129280 and c["M"] * c["N"] * c["K"] <= 4352 * 129280 * 4096:
                return c
    K = rng.choice([0, 1, 5, 16, 20, 32])
    T = round(rng.uniform(0.3, 2.0), 2)
    V = _log_int(rng, 64, 151936)
    if op == "logprobs":
        return {"op": op, "M": _log_int(rng, 1, min(4352, 4352 * 129280 // V)), "V": V, "pad": rng.choice([0, 0, 1, 24, 77]),
                "bf16": rng.random() < 0.5, "K": K, "T": T, "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    return {"op": op, "B": _log_int(rng, 1, 200), "L": rng.randint(1, 16), "V": V, "K": K, "T": T}


def _accepted(case):
    """Accepted lengths of the blocks: every length from 1 to L + 1 in turn (the order is the seed's)."""
    return [1 + (5 * b + 3) % (case["L"] + 1) for b in range(case["B"])]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["M"] * case["d"]
        read = 2 * n * (2 if case["residual"] else 1) + 2 * case["d"]
        written = (2 * n if case["residual"] else 0) + (n + 4 * case["M"] if case["i8"] else 2 * n)
        return {"bytes": read + written, "flops": 6 * n}
    if op == "quant":
        n = case["M"] * case["d"]
        return {"bytes": 3 * n + 4 * case["M"], "flops": 3 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + (2 if case["bf16"] else 4) * M * N, "flops": 2 * M * N * K}
    if op == "logprobs":
        rows, size = case["M"], 2 if case["bf16"] else 4
    else:
        rows, size = sum(_accepted(case)), 4
    return {"bytes": rows * (case["V"] * size + 20 + 8 * case["K"]), "flops": 6 * rows * case["V"]}


# --------------------------------------------------------------- inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _logits(g, rows, V, ld, dtype, masked):
    """Rows of logits as a language model has them: a wide body, a few tokens far above it, masked tokens at -inf."""
    z = torch.randn((rows, ld), generator=g, device="cuda") * 2.5
    z[:, :min(4, V)] += 9.0 * torch.rand((rows, min(4, V)), generator=g, device="cuda")
    if masked:
        z.masked_fill_(torch.rand((1, ld), generator=g, device="cuda") < masked, -math.inf)
    return z.to(dtype)


def _outputs(shape, K):
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    return {"logp": f(*shape), "rank": i(*shape), "entropy": f(*shape), "lse": f(*shape), "top_logp": f(*shape, K),
            "top_idx": i(*shape, K)}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        M, d = case["M"], case["d"]
        # hidden states with a few channels far larger than the others, as trained models have them
        wide = 1.0 + 15.0 * (torch.rand(d, generator=g, device="cuda") < 0.01).float()
        s["x"] = (_normal(g, (M, d)) * wide).bfloat16()
        s["residual"] = (_normal(g, (M, d), 3.0) * wide).bfloat16() if case["residual"] else None
        s["gamma"] = (1.0 + _normal(g, (d,), 0.2)).bfloat16()
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["i8"]:
            s["q"] = torch.empty((M, d), dtype=torch.int8, device="cuda")
            s["scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
        else:
            s["y"] = torch.empty_like(s["x"])
    elif op == "quant":
        M, d = case["M"], case["d"]
        s["x"] = _normal(g, (M, d), d ** -0.5).bfloat16()
        s["q"] = torch.empty((M, d), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        # rows as the quantisers leave them: bell-shaped, the largest value of a row near 127
        q = lambda r: torch.clamp(torch.round(torch.randn((r, K), generator=g, device="cuda") * 32.0), -127, 127).to(torch.int8)
        s["A"], s["Bw"] = q(M), q(N)
        s["sa"] = torch.rand(M, generator=g, device="cuda") * 0.02 + 0.01
        s["sb"] = (torch.rand(N, generator=g, device="cuda") * 0.02 + 0.01) * K ** -0.5
        s["C"] = torch.empty((M, N), dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    elif op == "logprobs":
        M, V = case["M"], case["V"]
        z = _logits(g, M, V, V + case["pad"], torch.bfloat16 if case["bf16"] else torch.float32, case["masked"])
        s["logits"] = z[:, :V]
        s["tokens"] = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["out"] = _outputs((M,), case["K"])
    else:
        B, L, V = case["B"], case["L"], case["V"]
        s["logits"] = _logits(g, B * (L + 1), V, V, torch.float32, 0.0)
        s["draft"] = torch.randint(0, V, (B, L), generator=g, device="cuda", dtype=torch.int32)
        order = torch.randperm(B, generator=g, device="cuda")
        s["accept_len"] = torch.tensor(_accepted(case), dtype=torch.int32, device="cuda")[order].contiguous()
        s["next_token"] = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["out"] = _outputs((B, L + 1), case["K"])
    return s


# ------------------------------------------------------------ one pass ---

def _plain_quantised(hg, r):
    """Rows hg (every value exact in 32 bits) -> q, scale.  q rounds 127 hg / max|hg|, in 64 bits so that a value halfway
    between two steps is seen as such."""
    a = hg.abs().amax(dim=1)
    a64 = torch.where(a > 0, a, torch.ones_like(a)).double()
    q = torch.round(127.0 * hg.double() / a64[:, None]).to(torch.int8)
    return q, a * r / 127.0


def _plain_logprobs(z, tokens, T, K):
    z = z.float()
    y = z / T
    m = y.amax(dim=1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)   # a row with every token masked: lse -inf, entropy 0
    e = torch.exp(y - m)
    total = e.sum(dim=1, dtype=torch.float64)
    dead = total == 0
    lse = m[:, 0].double() + torch.log(total)
    shift = torch.where(dead, torch.zeros_like(lse), lse)     # every token of such a row has -inf
    zt = torch.gather(z, 1, tokens.long()[:, None])
    logp = zt[:, 0].double() / T - shift
    # p * (y - m) is 0 where p is 0
    inner = torch.where(e > 0, e * (y - m), torch.zeros_like(e)).sum(dim=1, dtype=torch.float64) / total
    entropy = torch.where(dead, torch.zeros_like(lse), torch.log(total) - inner)
    rank = 1 + (z > zt).sum(dim=1)
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)   # equal values: the lower index first
    top = val[:, :K].double() / T - shift[:, None]
    return {"logp": logp.float(), "rank": rank.int(), "entropy": entropy.float(), "lse": lse.float(),
            "top_logp": top.float(), "top_idx": idx[:, :K].int()}


def _emitted_tokens(s):
    """(token of every row, whether the row was emitted) for the rows of the blocks, [B, L + 1] each."""
    B, L = s["draft"].shape
    i = torch.arange(L + 1, device="cuda")[None, :]
    n = s["accept_len"][:, None]
    drafted = torch.cat([s["draft"], s["draft"][:, :1]], dim=1)
    return torch.where(i == n - 1, s["next_token"][:, None], drafted), i < n


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        lib = _lib()
        if op == "norm":
            if case["i8"]:
                return lib.dflash_rmsnorm_i8(s["x"], s["gamma"], residual=s["residual"], eps=1e-6, q=s["q"],
                                             scale=s["scale"], h=s["h"])
            return lib.dflash_rmsnorm(s["x"], s["gamma"], residual=s["residual"], eps=1e-6, y=s["y"], h=s["h"])
        if op == "quant":
            return lib.dflash_quant_i8(s["x"], q=s["q"], scale=s["scale"])
        if op == "gemm":
            return lib.dflash_gemm_i8(s["A"], s["sa"], s["Bw"], s["sb"], C=s["C"], dev_status=s["status"])
        if op == "logprobs":
            return lib.dflash_token_logprobs(s["logits"], s["tokens"], K=case["K"], temperature=case["T"],
                                             dev_status=s["status"], **s["out"])
        return lib.dflash_emitted_logprobs(s["logits"], s["draft"], s["accept_len"], s["next_token"], K=case["K"],
                                           temperature=case["T"], dev_status=s["status"], **s["out"])
    if op == "norm":
        h = s["x"]
        if case["residual"]:
            h = (s["x"].float() + s["residual"].float()).bfloat16()
        f = h.float()
        r = torch.rsqrt(f.square().mean(dim=1) + 1e-6)
        hg = f * s["gamma"].float()
        out = _plain_quantised(hg, r) if case["i8"] else ((hg * r[:, None]).bfloat16(),)
        return (*out, h if case["residual"] else None)
    if op == "quant":
        x = s["x"].float()
        return _plain_quantised(x, torch.ones(x.shape[0], device=x.device))
    if op == "gemm":
        # sums of 8-bit products pass 2^24: in 64 bits they are exact
        c = s["A"].double() @ s["Bw"].double().t()
        return (c.float() * s["sa"][:, None] * s["sb"][None, :]).to(s["C"].dtype)
    if op == "logprobs":
        o = _plain_logprobs(s["logits"], s["tokens"], case["T"], case["K"])
    else:
        tokens, valid = _emitted_tokens(s)
        o = _plain_logprobs(s["logits"], tokens.reshape(-1), case["T"], case["K"])
        shape = valid.shape
        # rows behind the accepted ones keep what they held: zeros
        o = {k: torch.where(valid if v.dim() == 1 else valid[..., None], v.reshape(*shape, *v.shape[1:]), s["out"][k])
             for k, v in o.items()}
    return tuple(o[k] for k in ("logp", "rank", "entropy", "lse", "top_logp", "top_idx"))


# ---------------------------------------------------------- in 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "quant"):
        v = s["x"].double()
        h = None
        if op == "norm":
            if case["residual"]:
                v = v + s["residual"].double()
                h = v = v.to(torch.bfloat16).double()
            v = v / torch.sqrt((v * v).sum(dim=1, keepdim=True) / case["d"] + 1e-6) * s["gamma"].double()
            if not case["i8"]:
                return v, h
        scale = v.abs().max(dim=1).values / 127.0
        return (None, scale, h) if op == "norm" else (None, scale)
    if op == "gemm":
        return torch.mm(s["A"].double() * s["sa"].double().unsqueeze(1), (s["Bw"].double() * s["sb"].double().unsqueeze(1)).T)
    rows, V, K = s["logits"].shape[0], case["V"], case["K"]
    if op == "emitted":
        accept, nxt, draft = s["accept_len"].tolist(), s["next_token"].tolist(), s["draft"].tolist()
        L = case["L"]
        which = [b * (L + 1) + i for b, n in enumerate(accept) for i in range(n)]
        token = [nxt[b] if i == n - 1 else draft[b][i] for b, n in enumerate(accept) for i in range(n)]
    else:
        which, token = list(range(rows)), s["tokens"].tolist()
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    entropy, lse = torch.zeros_like(logp), torch.zeros_like(logp)
    top = torch.zeros((rows, K), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)
    for at in range(0, len(which), step):
        at_rows = torch.tensor(which[at:at + step], device="cuda")
        t = torch.tensor(token[at:at + step], device="cuda")
        y = s["logits"][at_rows].double() / case["T"]
        big = y.max(dim=1).values
        none = big == -math.inf
        lp = torch.where(none[:, None], -math.inf, torch.log_softmax(torch.where(none[:, None], 0.0, y), dim=1))
        p = lp.exp()
        logp[at_rows] = lp[torch.arange(len(t), device="cuda"), t]
        entropy[at_rows] = -torch.where(p > 0, p * lp, 0.0).sum(dim=1)
        lse[at_rows] = torch.where(none, -math.inf, big - lp.max(dim=1).values)
        if K:
            top[at_rows] = torch.topk(lp, K, dim=1).values
    if op == "emitted":
        shape = (case["B"], case["L"] + 1)
        logp, entropy, lse, top = logp.view(shape), entropy.view(shape), lse.view(shape), top.view(*shape, K)
    return logp, None, entropy, lse, top, None
