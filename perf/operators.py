"""Cases and plain forms of the operators that surround the W8A8 linears in a serving step.

Four operators of ``moe_gemm_absmax_b200.w8a8``:

  linear    ``linear_epilogue``: the online W8A8 linear with bias, activation and residual in its epilogue
  append    ``kv_append``: new tokens' keys and values into a paged cache, int8 with fp32 scales or bf16
  attend    ``paged_attention``: one new token a sequence over that cache
  logprobs  ``token_logprobs``: log probabilities of given tokens, entropy and the top alternatives

``own`` chooses what ``run`` does: the operators written out in elementary torch operations, or the
library's calls on the same inputs.
"""
import math

import torch

own = False

#: Activations of the linear, by the name that the library's ACT_* constants carry.
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # One token through a square-ish projection: what a single stream pays per layer, bound by latency.
        {"name": "linear m1 qkv", "op": "linear", "M": 1, "K": 2048, "N": 4096, "act": "none", "bias": True, "residual": False},
        # The dense MLP's down projection of a decode step for 8 streams, added to the residual stream.
        {"name": "linear m8 down", "op": "linear", "M": 8, "K": 17408, "N": 5120, "act": "none", "bias": False, "residual": True},
        # An odd batch with drafted tokens in it, between the decode and the prompt kernels.
        {"name": "linear m37 up", "op": "linear", "M": 37, "K": 5120, "N": 17408, "act": "gelu_tanh", "bias": True, "residual": False},
        # A prompt of 4096 tokens: the largest product.
        {"name": "linear m4096", "op": "linear", "M": 4096, "K": 5120, "N": 17408, "act": "silu", "bias": True, "residual": True},
        # The cache write of a decode step, 64 streams.
        {"name": "append t64 int8", "op": "append", "T": 64, "Hkv": 8, "D": 128, "page": 16, "cache": "int8"},
        # The cache write of a whole prompt batch.
        {"name": "append t4096 bf16", "op": "append", "T": 4096, "Hkv": 8, "D": 128, "page": 64, "cache": "bf16"},
        # One stream in the middle of an ordinary conversation: latency.
        {"name": "attend b1 l1000 bf16", "op": "attend", "B": 1, "len": 1000, "Hkv": 4, "G": 8, "D": 128, "page": 16, "cache": "bf16"},
        # A few streams of a long context, int8 cache.
        {"name": "attend b8 l32768 int8", "op": "attend", "B": 8, "len": 32768, "Hkv": 4, "G": 6, "D": 256, "page": 64, "cache": "int8"},
        # A full batch of ragged contexts.
        {"name": "attend b64 l8191 int8", "op": "attend", "B": 64, "len": 8191, "Hkv": 8, "G": 4, "D": 128, "page": 16, "cache": "int8"},
        # The head's logits of one token, with the alternatives that a client asks for.
        {"name": "logprobs m1", "op": "logprobs", "M": 1, "V": 131072, "k": 20, "dtype": "bf16", "masked": False},
        # The tokens of a scored prompt: an odd vocabulary whose rows start at any element, fp32 logits.
        {"name": "logprobs m100 fp32", "op": "logprobs", "M": 100, "V": 100003, "k": 5, "dtype": "fp32", "masked": True},
        # The largest scored batch.
        {"name": "logprobs m1024", "op": "logprobs", "M": 1024, "V": 131072, "k": 20, "dtype": "bf16", "masked": False},
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "append", "attend", "attend", "logprobs"))
    if op == "linear":
        K = 16 * _log_int(rng, 16, 17408 // 16)
        N = 8 * _log_int(rng, 32, 34816 // 8)
        M = _log_int(rng, 1, max(1, min(4096, 365_000_000_000 // (K * N))))
        return {"op": op, "M": M, "K": K, "N": N, "act": rng.choice(ACTS), "bias": rng.random() < 0.6,
                "residual": rng.random() < 0.6}
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, 4096), "Hkv": rng.choice((1, 2, 3, 4, 8)), "D": rng.choice((64, 128, 256)),
                "page": rng.choice((8, 16, 32, 64, 128)), "cache": rng.choice(("int8", "bf16"))}
    if op == "attend":
        B, Hkv, D = _log_int(rng, 1, 64), rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256))
        most = min(32768, 536_000_000 // (B * Hkv * D))
        return {"op": op, "B": B, "len": _log_int(rng, 1, most), "Hkv": Hkv, "G": rng.choice((1, 2, 3, 4, 6, 8, 12, 16)),
                "D": D, "page": rng.choice((8, 16, 32, 64, 128)), "cache": rng.choice(("int8", "bf16"))}
    V = _log_int(rng, 1000, 200000)
    return {"op": op, "M": _log_int(rng, 1, min(1024, 134_000_000 // V)), "V": V, "k": rng.choice((0, 1, 5, 20, 32)),
            "dtype": rng.choice(("bf16", "bf16", "fp32")), "masked": rng.random() < 0.3}


def _lengths(case):
    """Context lengths of the batch: the first is the longest, the others spread evenly below it."""
    n = [case["len"]]
    for i in range(1, case["B"]):
        n.append(1 + int((case["len"] - 1) * ((i * 0.6180339887498949) % 1.0)))
    return n


def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N + (4 * N if case["bias"] else 0)
                + (2 * M * N if case["residual"] else 0), "flops": 2 * M * N * K}
    if case["op"] == "append":
        n = 2 * case["T"] * case["Hkv"]
        return {"bytes": n * case["D"] * 2 + n * (case["D"] + 4 if case["cache"] == "int8" else 2 * case["D"]) + 8 * case["T"],
                "flops": 2 * n * case["D"]}
    if case["op"] == "attend":
        L = sum(_lengths(case))
        row = case["D"] + 4 if case["cache"] == "int8" else 2 * case["D"]
        H = case["Hkv"] * case["G"]
        return {"bytes": 2 * L * case["Hkv"] * row + 4 * case["B"] * H * case["D"], "flops": 4 * L * H * case["D"]}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["M"] * (case["V"] * size + 12 + 8 * case["k"]), "flops": 5 * case["M"] * case["V"]}


# ------------------------------------------------------------------ inputs

def _codes(n_rows, D, g):
    """int8 codes and fp32 scales of rows of normal values, each row with a loudness of its own."""
    x = torch.randn((n_rows, D), generator=g, device="cuda")
    x *= torch.exp(0.3 * torch.randn((n_rows, 1), generator=g, device="cuda"))
    s = x.abs().amax(dim=1) / 127.0
    return torch.clamp(torch.round(x / s[:, None]), -127, 127).to(torch.int8), s


def _cache(pages, Hkv, page, D, kind, g):
    """One side of a paged cache [pages, Hkv, page, D] and its scales [pages, Hkv, page] (None for bf16)."""
    rows = pages * Hkv * page
    c = torch.empty((rows, D), dtype=torch.int8 if kind == "int8" else torch.bfloat16, device="cuda")
    s = torch.empty(rows, device="cuda") if kind == "int8" else None
    step = (1 << 26) // D
    for r in range(0, rows, step):
        n = min(step, rows - r)
        if kind == "int8":
            c[r:r + n], s[r:r + n] = _codes(n, D, g)
        else:
            c[r:r + n] = torch.randn((n, D), generator=g, device="cuda").to(torch.bfloat16)
    return c.view(pages, Hkv, page, D), None if s is None else s.view(pages, Hkv, page)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        x = torch.randn((M, K), generator=g, device="cuda")
        x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 1000)]] *= 16.0   # outlier channels
        s["x"] = x.to(torch.bfloat16)
        w = 0.02 * torch.randn((N, K), generator=g, device="cuda")
        s["sw"] = w.abs().amax(dim=1) / 127.0
        s["qw"] = torch.clamp(torch.round(w / s["sw"][:, None]), -127, 127).to(torch.int8)
        s["bias_v"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["res"] = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
    elif case["op"] == "append":
        T, Hkv, D, page = case["T"], case["Hkv"], case["D"], case["page"]
        pages = -(-T // page) + 1
        s["k"] = torch.randn((T, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        s["v"] = torch.randn((T, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        s["kc"], s["ks"] = _cache(pages, Hkv, page, D, case["cache"], g)
        s["vc"], s["vs"] = _cache(pages, Hkv, page, D, case["cache"], g)
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    elif case["op"] == "attend":
        B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
        lens = _lengths(case)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1
        s["kc"], s["ks"] = _cache(pages, Hkv, page, D, case["cache"], g)
        s["vc"], s["vs"] = _cache(pages, Hkv, page, D, case["cache"], g)
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
        table = torch.full((B, max(need)), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        s["table"], s["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        s["q"] = torch.randn((B, Hkv * case["G"], D), generator=g, device="cuda").to(torch.bfloat16)
    else:
        M, V = case["M"], case["V"]
        x = 2.5 * torch.randn((M, V), generator=g, device="cuda")
        tokens = torch.randint(0, V, (M,), generator=g, device="cuda")
        if case["masked"]:   # what a grammar forbids
            off = torch.rand((M, V), generator=g, device="cuda") < 0.3
            off[torch.arange(M, device="cuda"), tokens] = False
            x.masked_fill_(off, -math.inf)
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["tokens"] = tokens.to(torch.int32)
    return s


# ------------------------------------------------------------------ one pass

def _scale(m):
    """m / 127, the quotient itself: a tensor over a plain number is multiplied by the number's rounded reciprocal."""
    return m / torch.full_like(m, 127.0)


def _linear(s):
    x = s["x"].float()
    sx = _scale(x.abs().amax(dim=1, keepdim=True))
    qx = torch.clamp(torch.round(x / torch.where(sx > 0, sx, 1.0)), -127, 127)
    v = (qx @ s["qw"].float().t()) * sx * s["sw"]
    if s["bias_v"] is not None:
        v = v + s["bias_v"]
    if s["act"] == "relu":
        v = torch.clamp(v, min=0)
    elif s["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif s["act"] == "gelu":
        v = 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    elif s["act"] == "gelu_tanh":
        v = v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(torch.bfloat16)


def _write(x, cache, scale, slots, page):
    at, off = slots // page, slots % page
    if scale is None:
        cache[at, :, off] = x
        return cache
    f = x.float()
    sc = _scale(f.abs().amax(dim=2))
    cache[at, :, off] = torch.clamp(torch.round(f / torch.where(sc > 0, sc, 1.0)[..., None]), -127, 127).to(torch.int8)
    scale[at, :, off] = sc
    return cache


def _held(cache, scale):
    """The values that a cache stands for."""
    return cache if scale is None else torch.mul(cache, scale[..., None])


def _gathered(cache, scale, table):
    x = cache[table].float()                                       # [B, pages, Hkv, page, D]
    if scale is not None:
        x = x * scale[table][..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)                  # [B, Hkv, tokens, D]


def _attend(s):
    B, Hkv, G, D = s["B"], s["Hkv"], s["G"], s["D"]
    table = s["table"].clamp(min=0).long()
    q = s["q"].float().view(B, Hkv, G, D)
    a = q @ _gathered(s["kc"], s["ks"], table).transpose(2, 3) * (1 / math.sqrt(D))
    seen = torch.arange(a.shape[3], device=a.device) < s["lens"][:, None, None, None]
    a = torch.where(seen, a, -math.inf)
    p = torch.exp(a - a.amax(dim=3, keepdim=True))
    y = (p @ _gathered(s["vc"], s["vs"], table)) / p.sum(dim=3, keepdim=True)
    return y.view(B, Hkv * G, D).to(torch.bfloat16)


def _logprobs(s):
    x = s["logits"].float()
    t = x - x.amax(dim=1, keepdim=True)
    e = torch.exp(t)
    z = e.sum(dim=1, keepdim=True)
    t = torch.where(e > 0, t, 0.0)
    entropy = torch.log(z) - (e * t).sum(dim=1, keepdim=True) / z
    lse = torch.log(z) + x.amax(dim=1, keepdim=True)
    out = {"logprob": (x.gather(1, s["tokens"].long()[:, None]) - lse)[:, 0], "entropy": entropy[:, 0]}
    if s["k"]:
        # descending, ties to the lower index: the value's bits in the order of values, then the index counted down
        b = (x + 0.0).view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = b * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
        ids = x.shape[1] - 1 - (torch.topk(key, s["k"], dim=1).values & 0xFFFFFFFF)
        out["top_ids"], out["top_logprobs"] = ids.to(torch.int32), x.gather(1, ids) - lse
    return out


def run(s):
    if own:
        from moe_gemm_absmax_b200 import w8a8
        if s["op"] == "linear":
            return w8a8.linear_epilogue(s["x"], s["qw"], s["sw"], bias=s["bias_v"], act=ACTS.index(s["act"]), residual=s["res"])
        if s["op"] == "append":
            w8a8.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], k_scale=s["ks"], v_scale=s["vs"])
            return [_held(s["kc"], s["ks"]), _held(s["vc"], s["vs"])]
        if s["op"] == "attend":
            return w8a8.paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"])
        logprob, entropy, ids, top = w8a8.token_logprobs(s["logits"], s["tokens"], topk=s["k"])
        out = {"logprob": logprob, "entropy": entropy}
        if s["k"]:
            out["top_ids"], out["top_logprobs"] = ids, top
        return out
    if s["op"] == "linear":
        return _linear(s)
    if s["op"] == "append":
        kc = _write(s["k"], s["kc"], s["ks"], s["slots"], s["page"])
        vc = _write(s["v"], s["vc"], s["vs"], s["slots"], s["page"])
        return [_held(kc, s["ks"]), _held(vc, s["vs"])]
    if s["op"] == "attend":
        return _attend(s)
    return _logprobs(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_linear(s):
    x = s["x"].double()
    # scale and quotient are fp32 numbers by definition, each correctly rounded: codes next to a border hang on them
    sx = (x.abs().max(dim=1).values / 127).float().double()[:, None]
    q = torch.where(sx > 0, (x / sx).float().double().round().clamp(-127, 127), 0.0)
    out = []
    for n in range(0, s["qw"].shape[0], 4096):
        out.append(torch.einsum("mk,nk->mn", q, s["qw"][n:n + 4096].double()) * s["sw"][n:n + 4096].double() * sx)
    v = torch.cat(out, dim=1)
    v = v if s["bias_v"] is None else v + s["bias_v"].double()
    f = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
         "gelu": lambda t: t * 0.5 * (1 + torch.erf(t / math.sqrt(2))),
         "gelu_tanh": lambda t: t * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))}[s["act"]]
    v = f(v)
    return v if s["res"] is None else v + s["res"].double()


def _exact_append(s):
    held = []
    for x, c, sc in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        c = c.double() if sc is None else c.double() * sc.double().unsqueeze(-1)
        x = x.double()
        if sc is not None:
            step = (x.abs().max(dim=-1, keepdim=True).values / 127).float().double()
            x = torch.where(step > 0, (x / step).float().double().round().clamp(-127, 127) * step, 0.0)
        for t, slot in enumerate(s["slots"].tolist()):
            c[slot // s["page"], :, slot % s["page"]] = x[t]
        held.append(c)
    return held


def _exact_attend(s):
    out = []
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, :-(-n // s["page"])].long()
        k, v = (c[ids].double() if sc is None else c[ids].double() * sc[ids].double().unsqueeze(-1)
                for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        k, v = (t.transpose(0, 1).reshape(s["Hkv"], -1, s["D"])[:, :n] for t in (k, v))
        q = s["q"][b].double().view(s["Hkv"], s["G"], s["D"])
        p = torch.softmax(torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(s["D"]), dim=2)
        out.append(torch.einsum("hgt,htd->hgd", p, v).reshape(-1, s["D"]))
    return torch.stack(out)


def _exact_logprobs(s):
    rows = []
    for x, tok in zip(s["logits"], s["tokens"].tolist()):
        lp = torch.log_softmax(x.double(), dim=0)
        order = torch.sort(x.float(), descending=True, stable=True).indices[:s["k"]]
        h = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum()
        rows.append((lp[tok], h, order.to(torch.int32), lp[order]))
    lp, h, ids, top = (torch.stack(c) for c in zip(*rows))
    out = {"logprob": lp, "entropy": h}
    if s["k"]:
        out["top_ids"], out["top_logprobs"] = ids, top
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](s)
