"""Cases of the operators around a paged cache of keys and values held in 4 bits: the table of a
step's rotations, appending a step's keys and values, attention over the cache, and reading it back.

`own` False: the plain forms, elementary torch operations in 32 bits.  `own` True: the calls of
q8_int8_block_gb300 that a serving program makes.

The cache is uint8 [pages, kv heads, page / 32, 36 d]: tiles of 32 tokens of one head.  Per tile the
keys' codes (16 d bytes), their scales (bfloat16 [d / 32][32 tokens]), the values' codes, their scales.
"""
import math
import random

import torch

own = False


# ---- the cases -----------------------------------------------------------------------------
def listed():
    tab = dict(op="table", axes=1, half=64, far=0)
    app = dict(op="append", heads=32, kv_heads=8, dim=128, rot=128, norm=True, f32=False, interleaved=False,
               batch=1, far=0, page=64, shape=1)
    att = dict(op="attention", heads=32, kv_heads=8, dim=128, new=1, page=64, shape=1)
    gat = dict(op="gather", kv_heads=8, dim=128, page=64, shape=1)
    return [
        # the rotations of one decode step of a serving batch; 64 of 256 channels turn
        dict(tab, name="table_step", tokens=64, half=32, far=100000),
        # a long prompt of text and images: time, height and width turn channels of their own
        dict(tab, name="table_image", tokens=8192, axes=3, far=30000),
        # the newest token of one request: latency counts
        dict(app, name="append_token", tokens=1, far=1000),
        # one token each of a serving batch, 256-wide heads of which 64 channels turn
        dict(app, name="append_batch", tokens=128, batch=128, far=4000, heads=16, kv_heads=4, dim=256, rot=64, shape=2),
        # a long prompt
        dict(app, name="append_prompt", tokens=8192),
        # packed prompts of odd lengths from binary32 projections, 64-wide heads without a norm
        dict(app, name="append_f32", tokens=2047, batch=5, heads=16, kv_heads=16, dim=64, rot=64, norm=False, f32=True,
             interleaved=True, far=77, page=32, shape=3),
        # the newest token of one request: latency counts
        dict(att, name="attention_one", batch=1, longest=1000),
        # a serving batch, contexts of very different lengths
        dict(att, name="attention_batch", batch=64, longest=8192, shape=2),
        # two requests about a book each
        dict(att, name="attention_long", batch=2, longest=131072, page=256, shape=3),
        # a few drafted tokens of every request checked at once, 256-wide heads
        dict(att, name="attention_verify", batch=16, longest=4097, new=5, heads=16, kv_heads=4, dim=256, shape=4),
        # the context of two requests for their next chunk of prompt
        dict(gat, name="gather_chunk", batch=2, longest=16384),
        # many short contexts of 64-wide heads
        dict(gat, name="gather_ragged", batch=16, longest=2001, kv_heads=16, dim=64, page=32, shape=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "append", "attention", "attention", "attention", "gather"])
    if op == "table":
        return dict(op=op, tokens=_log(rng, 1, 8192), axes=rng.choice([1, 1, 3]), half=rng.choice([16, 32, 64, 128]),
                    far=rng.choice([0, _log(rng, 10, 260000)]))
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([32, 64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    while heads > 32:
        heads -= kv
    more = dict(kv_heads=kv, dim=dim, page=page, shape=rng.randrange(1 << 20))
    if op == "append":
        tokens = _log(rng, 1, 4000)
        return dict(more, op=op, heads=heads, rot=rng.choice([dim, dim // 2, dim // 4]), norm=rng.random() < 0.6,
                    f32=rng.random() < 0.4, interleaved=rng.random() < 0.3, tokens=tokens,
                    batch=rng.choice([1, tokens, max(1, tokens // 300)]), far=rng.choice([0, _log(rng, 10, 4000)]))
    batch = _log(rng, 1, 128)
    longest = rng.choice([_log(rng, 1, 8192), _log(rng, 64, 131072)])
    while batch * longest * kv * dim > 1 << (28 if op == "attention" else 25):
        longest = max(1, longest // 2)
    if op == "gather":
        return dict(more, op=op, batch=batch, longest=longest)
    return dict(more, op=op, heads=heads, batch=batch, longest=longest, new=rng.choice([1, 1, 1, 2, 4, 7]))


def _lengths(case):
    """Tokens in the cache of each request: the longest, then lengths spread over its logarithm."""
    r = random.Random(case["shape"])
    n = [case["longest"]] + [max(1, int(case["longest"] ** r.random())) for _ in range(case["batch"] - 1)]
    r.shuffle(n)
    return n


def _new(case, n):
    """Each request's newest tokens, which ask."""
    r = random.Random(case["shape"] + 1)
    m = [min(x, case["new"] if x == case["longest"] else r.randint(1, case["new"])) for x in n]
    if case["new"] > 1 and len(m) > 6:
        m[3] = 0  # a request that asks nothing this time
    return m


def _runs(case):
    """append: (tokens before the new ones, new tokens) of each request."""
    r = random.Random(case["shape"])
    B, T = case["batch"], case["tokens"]
    cuts = list(range(T + 1)) if B == T else [0] + sorted(r.randint(0, T) for _ in range(B - 1)) + [T]
    return [(r.randint(0, case["far"]), b - a) for a, b in zip(cuts, cuts[1:])]


# ---- the cache's layout ----------------------------------------------------------------------
def _layout(d):
    """Where in a tile the bytes (channels 2 x and 2 x + 1) of its 32 tokens lie: keys, values [32, d / 2]."""
    tok = torch.arange(32, device="cuda")[:, None]
    c = torch.arange(0, d, 2, device="cuda")
    b, words = c // 32, min(4, d // 32)
    k = ((tok // 2 % 4 * max(1, d // 128) + b // 4) * 32 + (tok // 8 * 2 + tok % 2) * 4 + c % 32 // 8) * words
    k = (k + b % 4) * 4 + c % 8 // 2
    v = (tok % 8 * 32 + c % 32 // 4 * 4 + tok // 8) * (d // 64) + c // 64
    v = v * 4 + c % 64 // 32 * 2 + c % 4 // 2 + 18 * d
    return k, v


def _pages(lens, firsts, page, g):
    """(number of pages, block table): the pages of tokens firsts .. lens - 1 of each request, in no order."""
    need = [0 if n == 0 else (f + n - 1) // page - f // page + 1 for f, n in zip(firsts, lens)]
    total = sum(need) + 3  # some pages belong to nobody
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max([1] + [(f + n + page - 1) // page for f, n in zip(firsts, lens)])
    row = torch.arange(width, device="cuda")
    lo = torch.tensor([f // page for f in firsts], device="cuda")[:, None]
    cnt = torch.tensor(need, device="cuda")[:, None]
    at = (cnt.cumsum(0) - cnt) + (row - lo)
    bt = torch.where((row >= lo) & (row < lo + cnt), perm[at.clamp(0, total - 1)], -1)
    return total, bt.to(torch.int32).contiguous()


def _cum(v):
    return torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], device="cuda", dtype=torch.int32)


def _quantised(x):
    """Blocks of 32 along the last axis: the largest magnitude, and the codes -7 .. 7."""
    y = x.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    inv = torch.where(top < 2.0 ** -120, 0.0, torch.full_like(top, 7.0) / top)
    return top[..., 0], (y * inv).round().clamp_(-7, 7).flatten(-2)


def _bytes(codes):
    u = (codes + 8).to(torch.uint8)
    return u[..., 0::2] | u[..., 1::2] << 4


def _scale(top, r):
    return torch.where(top < 2.0 ** -120, 0.0, top * r * (1.0 / 7.0)).to(torch.bfloat16)


# ---- inputs --------------------------------------------------------------------------------
def _randn(g, *size):
    return torch.randn(*size, generator=g, device="cuda", dtype=torch.float32)


def _inv_freq(rot):
    return 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "table":
        T, half = case["tokens"], case["half"]
        s["inv_freq"] = _inv_freq(2 * half)
        if case["axes"] == 1:  # one token each of many requests, or a run behind a context
            t = torch.randint(0, case["far"] + 1, (T,), generator=g, device="cuda")
            s["positions"] = (t if T <= 128 else t[0] + torch.arange(T, device="cuda")).to(torch.int32)
            s["axis"] = None
        else:  # a text that goes on behind images; the axes' channels interleaved, time the rest
            t = torch.arange(T, device="cuda").repeat(3, 1) + case["far"]
            t[1:] -= torch.randint(0, 64, (2, T), generator=g, device="cuda")
            s["positions"] = t.clamp_(min=0).to(torch.int32)
            i = torch.arange(half, device="cuda", dtype=torch.int32)
            s["axis"] = torch.where(i < half * 3 // 4, i % 3, 0).to(torch.int32)
        return s
    Hk, d, page = case["kv_heads"], case["dim"], case["page"]
    s["lay"] = _layout(d)
    if case["op"] == "append":
        H, T = case["heads"], case["tokens"]
        runs = _runs(case)
        first, n = [a for a, _ in runs], [b for _, b in runs]
        # rows of the fused projection: queries, keys and values side by side; some channels are loud
        x = _randn(g, T, (H + 2 * Hk) * d) * torch.exp(0.3 * _randn(g, (H + 2 * Hk) * d))
        x = x if case["f32"] else x.to(torch.bfloat16)
        s["q"] = x[:, :H * d].view(T, H, d)
        s["k"] = x[:, H * d:(H + Hk) * d].view(T, Hk, d)
        s["v"] = x[:, (H + Hk) * d:].view(T, Hk, d)
        s["qw"], s["kw"] = (1.0 + 0.2 * _randn(g, d), 1.0 + 0.2 * _randn(g, d)) if case["norm"] else (None, None)
        s["first"] = torch.tensor(first, device="cuda", dtype=torch.int32)
        s["cu"] = _cum(n)
        tok = torch.arange(T, device="cuda", dtype=torch.int32)
        b = torch.searchsorted(s["cu"], tok, right=True) - 1
        pos = tok - s["cu"][b] + s["first"][b]
        total, s["block_table"] = _pages(n, first, page, g)
        s["slots"] = s["block_table"][b, pos // page] * page + pos % page
        turn = pos.double()[:, None] * _inv_freq(case["rot"])
        s["table"] = torch.stack((turn.cos(), turn.sin()), 1).float()
        s["cache"] = torch.zeros(total, Hk, page // 32, 36 * d, device="cuda", dtype=torch.uint8)
        return s
    n = _lengths(case)
    total, s["block_table"] = _pages(n, [0] * len(n), page, g)
    tiles = torch.empty(total * Hk * (page // 32), 36 * d, device="cuda", dtype=torch.uint8)
    for at, where in zip((0, 18 * d), s["lay"]):  # keys, values; some channels are loud
        x = _randn(g, total, Hk, page // 32, 32, d) * torch.exp(0.3 * _randn(g, Hk, 1, 1, d))
        top, codes = _quantised(x)
        tiles[:, where.flatten()] = _bytes(codes).view(tiles.shape[0], -1)
        tiles[:, at + 16 * d:at + 18 * d] = _scale(top, 1.0).transpose(-1, -2).contiguous().view(torch.uint8).view(tiles.shape[0], -1)
    s["cache"] = tiles.view(total, Hk, page // 32, 36 * d)
    if case["op"] == "gather":
        s["cu"], s["tokens"] = _cum(n), sum(n)
        return s
    m = _new(case, n)
    s["kv_len"] = torch.tensor(n, device="cuda", dtype=torch.int32)
    s["cu_q"] = _cum(m) if case["new"] > 1 else None
    s["most"] = max(m)
    s["q"] = (1.2 * _randn(g, sum(m), case["heads"], d)).to(torch.bfloat16)
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(s):
    if own:
        import q8_int8_block_gb300 as q8
        if s["op"] == "table":
            return q8.q8_rope_table(s["positions"], s["inv_freq"], axis=s["axis"])
        if s["op"] == "append":  # and the new tokens' keys and values as the cache holds them now
            q = q8.q8_kv4_append(s["k"], s["v"], s["cache"], s["slots"], table=s["table"], q=s["q"], q_weight=s["qw"],
                                 k_weight=s["kw"], eps=1e-6, interleaved=s["interleaved"])
            return q, q8.q8_kv4_gather(s["cache"], s["block_table"], s["cu"], s["tokens"], first=s["first"])
        if s["op"] == "gather":
            return q8.q8_kv4_gather(s["cache"], s["block_table"], s["cu"], s["tokens"])
        return q8.q8_kv4_attention(s["q"], s["cache"], s["block_table"], s["kv_len"], cu_q=s["cu_q"])
    return {"table": _plain_table, "append": _plain_append, "gather": _plain_gather, "attention": _plain_attention}[s["op"]](s)


def _plain_table(s):
    p = s["positions"] if s["axis"] is None else s["positions"][s["axis"].long()].T
    turn = (p[:, None] if s["axis"] is None else p).double() * s["inv_freq"]  # angles in 64 bits
    return torch.stack((turn.cos(), turn.sin()), 1).float()


def _turn(y, s):
    """The first rot channels of [T, heads, d] turned, each product and sum rounded to 32 bits."""
    rot = s["rot"]
    cos, sin = s["table"][:, 0, None], s["table"][:, 1, None]
    if s["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((z, y[..., rot:]), -1)


def _plain_append(s):
    d, page, cache = s["dim"], s["page"], s["cache"]

    def normed(x, w):
        x = x.float()
        if w is None:
            return x, 1.0
        return x * w, torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    q, r = normed(s["q"], s["qw"])
    q = _turn(q * r, s).to(torch.bfloat16)
    k, r = normed(s["k"], s["kw"])  # r goes into the scales
    slot = s["slots"].long()
    tile = cache.view(cache.shape[0], cache.shape[1], -1, cache.shape[-1])
    at = (slot // page, torch.arange(cache.shape[1], device=slot.device)[:, None], slot % page // 32)
    tok = slot % 32
    head = at[1].expand(-1, slot.shape[0]).T[..., None]
    pg, sub, blk = at[0][:, None, None], at[2][:, None, None], torch.arange(d // 32, device=slot.device)
    for x, f, where, off in ((_turn(k, s), r, s["lay"][0], 0), (s["v"].float(), 1.0, s["lay"][1], 18 * d)):
        top, codes = _quantised(x)
        tile[pg, head, sub, where[tok][:, None]] = _bytes(codes)
        two = _scale(top, f).unsqueeze(-1).view(torch.uint8)  # [T, kv heads, d / 32, 2 bytes]
        place = (off + 16 * d + 2 * (blk * 32 + tok[:, None]))[:, None, :, None] + torch.arange(2, device=slot.device)
        tile[pg[..., None], head[..., None], sub[..., None], place] = two
    return q, _plain_gather(s)


def _values(s):
    """What the whole cache stands for, 32 bits: keys and values [pages, kv heads, page, d]."""
    cache, d = s["cache"], s["dim"]
    tiles = cache.view(-1, 36 * d)
    out = []
    for where, off in zip(s["lay"], (0, 18 * d)):
        u = tiles[:, where.flatten()].view(-1, 32, d // 2)
        c = torch.stack((u & 15, u >> 4), -1).view(-1, 32, d // 32, 32).float() - 8.0
        sc = tiles[:, off + 16 * d:off + 18 * d].contiguous().view(torch.bfloat16).view(-1, d // 32, 32).float()
        out.append((c * sc.transpose(1, 2)[..., None]).view(cache.shape[0], cache.shape[1], s["page"], d))
    return out


def _plain_gather(s):
    cu, page = s["cu"].long(), s["page"]
    tok = torch.arange(s["tokens"], device=cu.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = tok - cu[b] + (s["first"][b] if "first" in s else 0)
    at = s["block_table"][b, pos // page].long()
    k, v = (x[at, :, pos % page].to(torch.bfloat16) for x in _values(s))
    return k, v


def _plain_attention(s):
    H, Hk, d, B = s["heads"], s["kv_heads"], s["dim"], s["batch"]
    bt, n = s["block_table"].long().clamp(min=0), s["kv_len"].long()
    dev, L = n.device, s["longest"]
    # the requests side by side, each padded to the longest
    k, v = (x[bt].transpose(1, 2).reshape(B, Hk, -1, d)[:, :, :L] for x in _values(s))
    cu = torch.arange(B + 1, device=dev) if s["cu_q"] is None else s["cu_q"].long()
    m, i = cu.diff(), torch.arange(s["most"], device=dev)
    q = s["q"][(cu[:-1, None] + i).clamp_(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, -1, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, d)
    hidden = torch.arange(L, device=dev) > (i + (n - m)[:, None])[:, :, None]
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hk, H // Hk, -1, L)
    x = x.masked_fill_(hidden[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    t = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, -1, L) @ v).view(B, Hk, H // Hk, -1, d) / t.masked_fill(t == 0.0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, H, d)
    tok = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu, tok, right=True) - 1
    return o[b, tok - cu[b]].to(torch.bfloat16)


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    if case["op"] == "table":
        n = case["tokens"] * case["half"]
        return {"bytes": 8 * n + 4 * case["tokens"] * case["axes"] + 8 * case["half"], "flops": 3 * n}
    Hk, d = case["kv_heads"], case["dim"]
    held = 2 * Hk * (d // 2 + d // 16)  # a token's bytes in the cache
    if case["op"] == "append":
        # inputs, rotations, rotated queries; the tokens' rows of the cache written, and read back as bfloat16
        H, T, e = case["heads"], case["tokens"], 4 if case["f32"] else 2
        return {"bytes": T * ((H + 2 * Hk) * d * e + 4 * case["rot"] + 2 * H * d + 2 * held + 4 * Hk * d),
                "flops": T * (4 * (H + Hk) * d + 3 * (H + Hk) * case["rot"] + 4 * 2 * Hk * d)}
    n = _lengths(case)
    if case["op"] == "gather":
        return {"bytes": sum(n) * (held + 4 * Hk * d), "flops": 4 * sum(n) * Hk * d}
    m = _new(case, n)
    H = case["heads"]
    seen = sum(a * b - a * (a - 1) // 2 for a, b in zip(m, n))
    return {"bytes": sum(b for a, b in zip(m, n) if a) * held + 4 * sum(m) * H * d, "flops": 4 * H * d * seen}


# ---- the definitions in 64 bits ----------------------------------------------------------------
def _held(s, b, n, values):
    """The first n tokens of request b as the cache holds them, 64 bits [n, kv heads, d], one token's place at a time."""
    d, page = s["dim"], s["page"]
    t = torch.arange(n, device="cuda")
    rows = s["cache"][s["block_table"][b].long()[t // page], :, t % page // 32].long()  # [n, kv heads, 36 d]
    t, c = (t % 32)[:, None], torch.arange(d, device="cuda")
    if values:  # channel 64 h + 32 e + 4 g + i in piece (token % 8, g, token / 8), word h, nibble 4 e + i
        word = (t % 8 * 32 + c % 32 // 4 * 4 + t // 8) * (d // 64) + c // 64
        nib, base = c % 64 // 32 * 4 + c % 4, 18 * d
    else:  # channel 32 b + 8 u + i in word (.., 2 (token / 8) + token % 2, u, b), nibble i
        w = min(4, d // 32)
        word = ((t // 2 % 4 * max(1, d // 128) + c // 128) * 32 + (t // 8 * 2 + t % 2) * 4 + c % 32 // 8) * w + c // 32 % 4
        nib, base = c % 8, 0
    pick = lambda i: torch.gather(rows, 2, i[:, None].expand(-1, rows.shape[1], -1))  # noqa: E731
    code = (pick(base + 4 * word + nib // 2) >> (nib % 2 * 4)) % 16 - 8
    at = base + 16 * d + 2 * (c // 32 * 32 + t)
    bits = (pick(at) + 256 * pick(at + 1)).to(torch.int32) << 16
    return code.double() * bits.view(torch.float32).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        p = s["positions"].double().view(-1, case["tokens"])
        axis = torch.zeros(case["half"], dtype=torch.long, device="cuda") if s["axis"] is None else s["axis"].long()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p[axis].T.contiguous() * s["inv_freq"])
        return torch.stack((turn.real, turn.imag), 1)
    d = case["dim"]
    if case["op"] == "append":
        h = case["rot"] // 2
        turn = torch.complex(s["table"][:, 0].double(), s["table"][:, 1].double())[:, None]

        def rotated(x, w):
            x = x.double()
            r = 1.0
            if w is not None:
                r = 1.0 / (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
                x = x * w.double()
            y = x[..., :2 * h].unflatten(-1, (h, 2) if case["interleaved"] else (2, h))
            y = y if case["interleaved"] else y.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            return torch.cat((z.flatten(-2), x[..., 2 * h:]), -1), r

        def held(x, r):  # blocks of 32: the codes by their definition, which rounds 7 / top and the products to 32 bits
            y = x.unflatten(-1, (-1, 32))
            top = y.abs().amax(-1, keepdim=True).float().double().clamp_min(1e-30)
            code = (y * (7.0 / top).float().double()).float().double().round()
            return (code * top / 7.0).flatten(-2) * r

        q, r = rotated(s["q"], s["qw"])
        return q * r, (held(*rotated(s["k"], s["kw"])), held(s["v"].double(), 1.0))
    n = _lengths(case)
    if case["op"] == "gather":
        return tuple(torch.cat([_held(s, b, x, v) for b, x in enumerate(n)]) for v in (False, True))
    G, out, cu = case["heads"] // case["kv_heads"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (x, m) in enumerate(zip(n, _new(case, n))):
        if not m:
            continue
        k, v = _held(s, b, x, False), _held(s, b, x, True)
        seen = torch.ones(m, x, dtype=torch.bool, device="cuda").tril(x - m)
        for h in range(case["kv_heads"]):
            q = s["q"][cu:cu + m, h * G:(h + 1) * G].double()
            w = torch.einsum("ngd,md->gnm", q, k[:, h]) / math.sqrt(d)
            w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
            out[cu:cu + m, h * G:(h + 1) * G] = torch.einsum("gnm,md->ngd", w, v[:, h])
        cu += m
    return out
