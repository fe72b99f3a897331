"""Cases of the attention layer's operators: heads' norm with rotation, attention over packed
prompts, and decode attention of a batch behind a shared prefix.

`own` False: the plain forms, elementary torch operations in 32 bits.  `own` True: the calls of
q8_int8_block_gb300 that a serving program makes.
"""
import math
import random

import torch

own = False


# ---- the cases -----------------------------------------------------------------------------
def listed():
    prompt = dict(op="prompt", heads=32, kv_heads=8, dim=128, fused=True, context=0, shape=1)
    qk = dict(op="qk", heads=32, kv_heads=8, dim=128, rot=128, f32=False, interleaved=False, far=0)
    pre = dict(op="prefix", heads=32, kv_heads=8, dim=128, head_major=False, shape=1)
    return [
        # one short question to a chat model: latency counts
        dict(prompt, name="prompt_short", batch=1, longest=77),
        # a whole document as one prompt
        dict(prompt, name="prompt_long", batch=1, longest=8192),
        # a serving batch: sixteen prompts of very different lengths packed behind one another
        dict(prompt, name="prompt_packed", batch=16, longest=2000, shape=5),
        # chunked prefill: up to 512 new tokens behind 16K that are cached already
        dict(prompt, name="prompt_chunk", batch=2, longest=512, context=16384, fused=False, shape=3),
        # 64-wide heads, every query head with a key head of its own
        dict(prompt, name="prompt_heads64", batch=4, longest=1531, heads=16, kv_heads=16, dim=64, shape=2),
        # the newest token of one request
        dict(qk, name="qk_token", tokens=1, far=30000),
        # a long prompt, straight from the binary32 outputs of the projection
        dict(qk, name="qk_prompt", tokens=8192, f32=True),
        # 256-wide heads of which 64 channels turn, odd number of tokens, behind a long context
        dict(qk, name="qk_wide", tokens=2047, heads=16, kv_heads=4, dim=256, rot=64, far=260000),
        # one token each of 64 requests, pairs side by side
        dict(qk, name="qk_batch", tokens=64, heads=20, kv_heads=4, dim=64, rot=64, interleaved=True, far=100000),
        # one request behind a short system prompt: latency counts
        dict(pre, name="prefix_one", batch=1, prefix=1000, longest=77),
        # a serving batch behind a long instruction, answers of very different lengths
        dict(pre, name="prefix_batch", batch=64, prefix=8192, longest=512, shape=2),
        # few requests about one book
        dict(pre, name="prefix_long", batch=8, prefix=131072, longest=256, head_major=True, shape=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "qk", "prefix", "prefix"])
    if op == "qk":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), f32=rng.random() < 0.4,
                    interleaved=rng.random() < 0.3, far=rng.choice([0, _log(rng, 10, 260000)]),
                    tokens=_log(rng, 1, 4000))
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    while heads > 32:
        heads -= kv
    if op == "prefix":
        batch = _log(rng, 1, 128)
        return dict(op=op, heads=heads, kv_heads=kv, dim=dim, batch=batch,
                    prefix=rng.choice([0, _log(rng, 1, 8192), _log(rng, 64, 131072 // batch)]),
                    longest=_log(rng, 1, 1024), head_major=rng.random() < 0.5, shape=rng.randrange(1 << 20))
    batch = _log(rng, 1, 16)
    context = rng.choice([0, 0, _log(rng, 1, 16000)])
    longest = _log(rng, 1, 4000)
    while batch * heads * longest * (longest + context) > (1 << 30):  # the plain form's scores
        longest = max(1, longest // 2)
        batch = max(1, batch - 1)
    return dict(op=op, heads=heads, kv_heads=kv, dim=dim, batch=batch, longest=longest, context=context,
                fused=context == 0 and rng.random() < 0.5, shape=rng.randrange(1 << 20))


def _lengths(case):
    """The lengths of a ragged batch: the longest, then lengths spread over its logarithm."""
    r = random.Random(case["shape"])
    n = [case["longest"]] + [int(case["longest"] ** r.random()) for _ in range(case["batch"] - 1)]
    if case["batch"] > 6:
        n[3] = 0  # a request that brings nothing this time
    r.shuffle(n)
    return n


def _contexts(case, n):
    """Tokens cached before each sequence's new ones."""
    r = random.Random(case["shape"] + 1)
    return [case["context"] if x == max(n) else int(case["context"] * r.random()) for x in n]


# ---- inputs --------------------------------------------------------------------------------
def _randn(g, *size):
    return torch.randn(*size, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H, Hk, d = case["heads"], case["kv_heads"], case["dim"]
    s = dict(case)
    if case["op"] == "qk":
        T = case["tokens"]
        # rows of the fused projection: queries, keys and values side by side; some channels are loud
        gain = torch.exp(0.5 * _randn(g, (H + 2 * Hk) * d))
        x = _randn(g, T, (H + 2 * Hk) * d) * gain
        x = x if case["f32"] else x.to(torch.bfloat16)
        s["q"] = x[:, :H * d].view(T, H, d)
        s["k"] = x[:, H * d:(H + Hk) * d].view(T, Hk, d)
        s["qw"], s["kw"] = 1.0 + 0.2 * _randn(g, d), 1.0 + 0.2 * _randn(g, d)
        # packed requests that begin at places of their own: one new token each, or runs of 500
        t, run_of = torch.arange(T, device="cuda"), 1 if T <= 128 else 500
        start = torch.randint(0, case["far"] + 1, (T // run_of + 1,), generator=g, device="cuda")
        s["positions"] = (t % run_of + start[t // run_of]).to(torch.int32)
        s["inv_freq"] = 1e6 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        return s
    n = _lengths(case)
    if case["op"] == "prompt":
        m = [a + b for a, b in zip(n, _contexts(case, n))] if case["context"] else n
        cum = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], device="cuda", dtype=torch.int32)  # noqa: E731
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = cum(n), cum(m), max(n), max(m)
        Tq, Tk = sum(n), sum(m)
        if case["fused"]:  # views of the projection's rows
            x = _randn(g, Tq, (H + 2 * Hk) * d).to(torch.bfloat16)
            s["q"] = x[:, :H * d].view(Tq, H, d)
            s["k"] = x[:, H * d:(H + Hk) * d].view(Tq, Hk, d)
            s["v"] = x[:, (H + Hk) * d:].view(Tq, Hk, d)
        else:
            s["q"] = _randn(g, Tq, H, d).to(torch.bfloat16)
            s["k"] = _randn(g, Tk, Hk, d).to(torch.bfloat16)
            s["v"] = _randn(g, Tk, Hk, d).to(torch.bfloat16)
        return s
    B, P, cap = case["batch"], case["prefix"], case["longest"]
    s["q"] = _randn(g, B, H, d).to(torch.bfloat16)
    if case["head_major"]:  # caches with each head's keys behind one another
        mk = lambda *lead: [_randn(g, *lead[:-1], Hk, lead[-1], d).to(torch.bfloat16).transpose(-3, -2) for _ in range(2)]  # noqa: E731
    else:
        mk = lambda *lead: [_randn(g, *lead, Hk, d).to(torch.bfloat16) for _ in range(2)]  # noqa: E731
    s["k_prefix"], s["v_prefix"] = mk(P)
    s["k_own"], s["v_own"] = mk(B, cap)
    s["own_len"] = torch.tensor(n, device="cuda", dtype=torch.int32)
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(s):
    if own:
        import q8_int8_block_gb300 as q8
        if s["op"] == "qk":
            return q8.q8_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["qw"],
                                      k_weight=s["kw"], eps=1e-6, interleaved=s["interleaved"])
        if s["op"] == "prompt":
            return q8.q8_prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
        return q8.q8_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_own"], s["v_own"], s["own_len"])
    return {"qk": _plain_qk, "prompt": _plain_prompt, "prefix": _plain_prefix}[s["op"]](s)


def _plain_qk(s):
    # angles of far positions in 64 bits, the rest in 32
    t = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin, rot = t.cos().float(), t.sin().float(), s["rot"]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        y, rest = x[..., :rot], x[..., rot:]
        if s["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((y, rest), -1).to(torch.bfloat16)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _softmax(x):
    """Weights without their sum, and the sum; a row of -inf gives zeros."""
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    t = x.sum(-1, keepdim=True)
    return x, t.masked_fill(t == 0.0, 1.0)


def _plain_prompt(s):
    # the sequences side by side, each padded to the longest
    cu_q, cu_k, L, M = s["cu_q"].long(), s["cu_k"].long(), s["max_q"], s["max_k"]
    H, Hk, d, B = s["heads"], s["kv_heads"], s["dim"], s["batch"]
    dev, Tq, Tk = cu_q.device, s["q"].shape[0], s["k"].shape[0]
    iq, ik = torch.arange(L, device=dev), torch.arange(M, device=dev)
    lq, lk = cu_q.diff(), cu_k.diff()
    q = s["q"][(cu_q[:-1, None] + iq).clamp_(max=Tq - 1)].float()
    at = (cu_k[:-1, None] + ik).clamp_(max=Tk - 1)
    k, v = s["k"][at].float().permute(0, 2, 3, 1), s["v"][at].float().permute(0, 2, 1, 3)
    q = q.view(B, L, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, H // Hk * L, d)
    hidden = ik > (iq + (lk - lq)[:, None])[:, :, None]
    x = (q @ k).mul_(1.0 / math.sqrt(d)).view(B, Hk, H // Hk, L, M).masked_fill_(hidden[:, None, None], -math.inf)
    p, t = _softmax(x)
    o = ((p.view(B, Hk, -1, M) @ v).view(B, Hk, -1, L, d) / t).permute(0, 3, 1, 2, 4).reshape(B, L, H, d)
    tok = torch.arange(Tq, device=dev)
    b = torch.searchsorted(cu_q, tok, right=True) - 1
    return o[b, tok - cu_q[b]].to(torch.bfloat16)


def _plain_prefix(s):
    H, Hk, d, B, P = s["heads"], s["kv_heads"], s["dim"], s["batch"], s["prefix"]
    q = s["q"].float().view(B, Hk, H // Hk, d)
    # [Hk, B G, d] x [Hk, d, P]: the shared keys for all requests at once
    x = (q.transpose(0, 1).reshape(Hk, -1, d) @ s["k_prefix"].float().permute(1, 2, 0)).view(Hk, B, -1, P).transpose(0, 1)
    y = q @ s["k_own"].float().permute(0, 2, 3, 1)
    hidden = torch.arange(y.shape[-1], device=y.device) >= s["own_len"][:, None]
    x = torch.cat((x, y.masked_fill_(hidden[:, None, None], -math.inf)), -1).mul_(1.0 / math.sqrt(d))
    p, t = _softmax(x)
    o = (p[..., :P].transpose(0, 1).reshape(Hk, -1, P) @ s["v_prefix"].float().transpose(0, 1)).view(Hk, B, -1, d).transpose(0, 1)
    o = o + p[..., P:] @ s["v_own"].float().transpose(1, 2)
    return (o / t).reshape(B, H, d).to(torch.bfloat16)


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    H, Hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        T = case["tokens"]
        n = T * (H + Hk) * d
        # square and sum, two scalings, and the rotation's four products and two sums a pair
        return {"bytes": n * (4 if case["f32"] else 2) + 2 * n + 4 * T + 8 * d + 4 * case["rot"],
                "flops": 4 * n + 3 * T * (H + Hk) * case["rot"]}
    n = _lengths(case)
    if case["op"] == "prompt":
        c = _contexts(case, n) if case["context"] else [0] * len(n)
        seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, c))
        return {"bytes": 2 * d * (2 * H * sum(n) + 2 * Hk * (sum(n) + sum(c))), "flops": 4 * H * d * seen}
    B, P = case["batch"], case["prefix"]
    return {"bytes": 2 * d * (2 * H * B + 2 * Hk * (P + sum(n))), "flops": 4 * H * d * (B * P + sum(n))}


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double().outer(s["inv_freq"]))[:, None]
        out = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            x = x / (x.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * w.double()
            h = case["rot"] // 2
            y = x[..., :2 * h].unflatten(-1, (h, 2) if case["interleaved"] else (2, h))
            y = y if case["interleaved"] else y.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            out.append(torch.cat((z.flatten(-2), x[..., 2 * h:]), -1))
        return tuple(out)
    G, r = case["heads"] // case["kv_heads"], 1.0 / math.sqrt(case["dim"])

    def attend(q, k, v, seen):
        """q [n, H, d], k and v [m, Hk, d], seen [n, m]: one head group at a time."""
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for h in range(k.shape[1]):
            x = torch.einsum("ngd,md->gnm", q[:, h * G:(h + 1) * G].double(), k[:, h].double()) * r
            x = x.masked_fill(~seen, -math.inf)
            if x.shape[-1]:
                o[:, h * G:(h + 1) * G] = torch.einsum("gnm,md->ngd", torch.softmax(x, -1).nan_to_num(0.0), v[:, h].double())
        return o

    if case["op"] == "prompt":
        a, b, parts = s["cu_q"].tolist(), s["cu_k"].tolist(), []
        for i in range(case["batch"]):
            n, m = a[i + 1] - a[i], b[i + 1] - b[i]
            seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
            parts.append(attend(s["q"][a[i]:a[i + 1]], s["k"][b[i]:b[i + 1]], s["v"][b[i]:b[i + 1]], seen))
        return torch.cat(parts)
    parts = []
    for i, n in enumerate(s["own_len"].tolist()):
        k, v = (torch.cat((s[x + "_prefix"], s[x + "_own"][i, :n])) for x in ("k", "v"))
        parts.append(attend(s["q"][i:i + 1], k, v, torch.ones(1, k.shape[0], dtype=torch.bool, device="cuda")))
    return torch.cat(parts)
