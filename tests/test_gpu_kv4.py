"""The paged 4-bit cache: append, gather and attention against the plain forms of
tests/kv4_ref.py, which derives the tolerances; the table of rotations against binary64."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402
from tests import kv4_ref as K  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN16 = 0x7FC0


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


def i32(x):
    return torch.tensor(x, device="cuda", dtype=I32)


def cum(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


# ---- table -------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,half,far", [(1, 8, 0), (1, 64, 260000), (7, 32, 2 ** 31 - 8), (300, 128, 1000), (5000, 64, 100000)])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_table(q8, T, half, far, axes):
    inv = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    pos = torch.arange(T, device="cuda", dtype=torch.int64) + far
    axis = None
    if axes:
        pos = torch.stack([pos, pos // 3, pos % 17][:axes])
        axis = torch.arange(half, device="cuda", dtype=I32) % axes
    got = q8.q8_rope_table(pos.to(I32), inv, axis=axis)
    assert got.shape == (T, 2, half) and got.dtype == F32
    angle = (pos[:, None] if axis is None else pos[axis.long()].T).double() * inv
    ref = torch.stack((angle.cos(), angle.sin()), 1)
    # the angle to 2^-31 turns (2^-28 rad) and its own rounding, at most an eighth of a turn (2^-25 rad,
    # and 2^-25 for pi), sine and cosine to two roundings; the reference's product to 2^-53 of it
    tol = 2.0 ** -28 + 2.0 ** -24 + 2.0 ** -23 + angle.abs()[:, None] * 2.0 ** -52
    R.assert_within(got, ref, tol.expand_as(ref), "table")
    assert q8.q8_device_error() == 0


def test_table_marks_what_has_no_angle(q8):
    inv = torch.tensor([1.0, 2.0 ** 32, math.inf, math.nan, -0.5, 0.0, 1.0, 1.0], device="cuda", dtype=torch.float64)
    axis = i32([0, 0, 0, 0, 0, 0, 2, -1])
    got = q8.q8_rope_table(i32([[3, -7]]), inv, axis=axis)
    bad = torch.tensor([0, 1, 1, 1, 0, 0, 1, 1], device="cuda").bool()
    assert got[..., bad].isnan().all() and not got[..., ~bad].isnan().any()
    assert torch.equal(got[:, :, 5], torch.tensor([[1.0, 0.0]] * 2, device="cuda"))
    R.assert_within(got[:, 1, 4], torch.tensor([-1.5, 3.5], device="cuda", dtype=torch.float64).sin(),
                    torch.full((2,), 2.0 ** -22, device="cuda", dtype=torch.float64))


# ---- append ------------------------------------------------------------------------------------
def fused_rows(T, H, Hkv, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, (H + 2 * Hkv) * d, generator=g, device="cuda") *
         torch.exp(torch.randn((H + 2 * Hkv) * d, generator=g, device="cuda"))).to(dtype)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    return x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hkv) * d].view(T, Hkv, d), x[:, (H + Hkv) * d:].view(T, Hkv, d), w


def table_of(T, rot, seed=0):
    if rot == 0:
        return None
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.rand(T, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 6.283
    return torch.stack((a.cos(), a.sin()), 1).float()


def check_cache(cache, before, slots, k, v, kw, table, interleaved, page, eps=1e-6):
    """The bytes of the cache: codes bit for bit, scales bit for bit (keys with a norm: within a step),
    everything else as it was."""
    pages, Hkv, tiles, _ = cache.shape
    d = k.shape[2]
    put = [t for t, s in enumerate(slots) if 0 <= s < pages * page]
    kc, ktop = K.quantised(K.turned(k.cpu(), None if kw is None else kw.cpu(), None if table is None else table.cpu(), interleaved))
    vc, vtop = K.quantised(v.cpu().float())
    r = torch.ones(()) if kw is None else 1.0 / (k.cpu().double().square().mean(-1, keepdim=True) + eps).sqrt()
    want = [x.clone() for x in K.unpack(before.reshape(-1, 36 * d))]
    got = K.unpack(cache.reshape(-1, 36 * d))
    sc = [(ktop.double() * r * (1.0 / 7.0)).float().to(BF16), (vtop * torch.tensor(1.0 / 7.0)).to(BF16)]
    for t in put:
        s = slots[t]
        rows = (s // page * Hkv + torch.arange(Hkv)) * tiles + s % page // 32
        for x, y in zip(want, (kc, vc, *sc)):
            x[rows, s % 32] = y[t].to(x.dtype)
    for i, name in enumerate(("key codes", "value codes", "key scales", "value scales")):
        if i == 2 and kw is not None:
            off = (got[i].view(torch.int16).int() - want[i].view(torch.int16).int()).abs()
            assert int(off.max()) <= 1, name
        elif i >= 2:
            assert torch.equal(got[i].view(torch.int16), want[i].view(torch.int16)), name
        else:
            assert torch.equal(got[i], want[i]), name


def check_q(out, q, w, table, interleaved, eps=1e-6):
    x = q.double().cpu()
    r = 1.0 if w is None else 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    z = K.turned(q.cpu(), None, None, False).double() * (1.0 if w is None else w.cpu().double())
    ref, size = z.clone(), z.abs()
    if table is not None:
        half = table.shape[2]
        cos, sin = table[:, 0, None].cpu().double(), table[:, 1, None].cpu().double()
        i = torch.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = z[..., ia], z[..., ib]
        ref[..., ia], ref[..., ib] = a * cos - b * sin, a * sin + b * cos
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    # binary32: (d / 2 + 12) 2^-24 relative of the terms, below 2^-16; then one rounding to bfloat16
    R.assert_within(out.cpu(), ref * r, K.STEP * (ref * r).abs() * (1 + 2.0 ** -7) + size * r * 2.0 ** -16, "queries")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,Hkv,d,rot,page,norm", [
    (1, 32, 8, 128, 128, 64, True), (1, 1, 1, 64, 64, 32, False), (2, 5, 5, 64, 32, 32, True), (33, 12, 4, 256, 64, 96, True),
    (7, 3, 3, 128, 0, 64, True), (5, 0, 2, 128, 96, 128, True), (3, 4, 0, 64, 16, 32, True), (65, 7, 1, 256, 256, 256, False),
    (40, 3, 3, 64, 48, 64, False), (700, 9, 3, 128, 64, 64, True)])
def test_append(q8, T, H, Hkv, d, rot, page, norm, dtype, interleaved):
    q, k, v, (qw, kw) = fused_rows(T, H, Hkv, d, dtype, seed=T + d)
    qw, kw = (qw, kw) if norm else (None, None)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].tolist()
    slots[T // 2] = -1 - T
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, q8.q8_kv4_cache_shape(pages, page, Hkv, d), generator=g, device="cuda", dtype=torch.uint8)
    before, table = cache.clone(), table_of(T, rot)
    out = q8.q8_kv4_append(k, v, cache, i32(slots), table=table, q=q if H else None, q_weight=qw, k_weight=kw,
                           interleaved=interleaved)
    assert q8.q8_device_error() == 0
    if Hkv:
        check_cache(cache, before, slots, k, v, kw, table, interleaved, page)
    if H:
        assert out.dtype == BF16 and out.is_contiguous()
        check_q(out, q, qw, table, interleaved)
    else:
        assert out is None
    again = cache.clone()
    out2 = q8.q8_kv4_append(k, v, cache, i32(slots), table=table, q=q if H else None, q_weight=qw, k_weight=kw,
                            interleaved=interleaved)
    assert torch.equal(again, cache) and (out is None or torch.equal(out, out2))


@pytest.mark.parametrize("dtype,interleaved", [(BF16, False), (F32, True)])
@pytest.mark.parametrize("runs,H,Hkv,d,rot,page", [
    ([(0, 2050)], 4, 16, 128, 128, 64), ([(77, 700), (5, 1), (31, 33), (64, 320)], 2, 64, 64, 32, 32),
    ([(13, 1500), (200, 31)], 0, 20, 256, 64, 96), ([(1, 999)], 3, 31, 128, 0, 256), ([(3, 500)], 2, 3, 128, 64, 64)])
def test_append_of_many_tokens(q8, runs, H, Hkv, d, rot, page, dtype, interleaved):
    """Packed prompts whose pages lie anywhere: neighbours that end in one tile and go on in another, tiles
    written in part, tokens that are not kept, and slots in no order at all."""
    T = sum(n for _, n in runs)
    q, k, v, (qw, kw) = fused_rows(T, H, Hkv, d, dtype, seed=T)
    need = [-(-(a + n) // page) for a, n in runs]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(T)).tolist()
    slots, at = [], 0
    for (a, n), m in zip(runs, need):
        slots += [perm[at + t // page] * page + t % page for t in range(a, a + n)]
        at += m
    table = table_of(T, rot)
    for case in ("runs", "holes", "anywhere"):
        if case == "holes":
            slots[40], slots[100:140], slots[T - 1] = -1, [-5] * 40, pages * page
        elif case == "anywhere":
            slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].tolist()
        g = torch.Generator(device="cuda").manual_seed(1)
        cache = torch.randint(0, 256, q8.q8_kv4_cache_shape(pages, page, Hkv, d), generator=g, device="cuda", dtype=torch.uint8)
        before = cache.clone()
        out = q8.q8_kv4_append(k, v, cache, i32(slots), table=table, q=q if H else None, q_weight=qw if H else None,
                               k_weight=kw, interleaved=interleaved)
        assert q8.q8_device_error() == (1 << 10 if case == "holes" else 0)
        check_cache(cache, before, slots, k, v, kw, table, interleaved, page)
        if H:
            check_q(out, q, qw, table, interleaved)


def test_append_of_zeros_ties_and_extremes(q8):
    d, page = 128, 32
    x = torch.zeros(6, 1, d, device="cuda")
    x[1] = 2.0 ** -126            # below 2^-120: zeros
    x[2] = 2.0 ** -119
    x[3] = torch.linspace(-7, 7, d, device="cuda") * 2.0 ** 100
    x[4] = (torch.arange(d, device="cuda") % 15 - 7).float()
    x[4] += 0.5                   # ties, to the even code
    x[4, 0, ::32] = 7.0
    x[5] = 3.4e38
    cache = torch.zeros(q8.q8_kv4_cache_shape(1, page, 1, d), device="cuda", dtype=torch.uint8)
    before, slots = cache.clone(), [3, 0, 31, 8, 9, 10]
    q8.q8_kv4_append(x, x, cache, i32(slots))
    check_cache(cache, before, slots, x, x, None, None, False, page)
    bt, cu = i32([[0]]), i32([0, 32])
    k, v = q8.q8_kv4_gather(cache, bt, cu, 32, out_dtype=F32)
    assert torch.equal(k[3], torch.zeros_like(k[3])) and torch.equal(k[0], torch.zeros_like(k[0]))
    assert torch.equal(k, v) and bool(torch.isfinite(k).all())


@pytest.mark.parametrize("T", [5, 4800])  # a warp a token; tiles through shared memory
@pytest.mark.parametrize("dtype,odd", [(BF16, math.nan), (BF16, -math.inf), (F32, math.nan), (F32, math.inf)])
def test_append_keeps_what_is_not_finite(q8, T, dtype, odd):
    H, Hkv, d, page = 2, 8, 128, 64
    assert T < 100 or T * Hkv * d >= 24576 * torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v, _ = fused_rows(T, H, Hkv, d, dtype, seed=1)
    q, k, v = q.clone(), k.clone(), v.clone()
    slots, bt, cu = i32(list(range(T))), i32([list(range(-(-T // page)))]), i32([0, T])
    caches = [torch.zeros(q8.q8_kv4_cache_shape(-(-T // page), page, Hkv, d), device="cuda", dtype=torch.uint8) for _ in range(2)]
    table = table_of(T, 32)
    clean = q8.q8_kv4_append(k, v, caches[0], slots, table=table, q=q)
    k[1, 3, 70], v[2, 7, 5], k[4, 0, 3], q[3, 1, 100], q[0, 0, 2] = odd, odd, odd, odd, odd
    out = q8.q8_kv4_append(k, v, caches[1], slots, table=table, q=q)
    rows = [q8.q8_kv4_gather(c, bt, cu, T, out_dtype=F32) for c in caches]
    where = [torch.zeros(T, Hkv, d, device="cuda", dtype=torch.bool) for _ in range(2)]
    where[0][1, 3, 64:96], where[0][4, 0, :32], where[1][2, 7, :32] = True, True, True  # whole blocks
    for i in range(2):
        assert not rows[1][i][where[i]].isfinite().any()
        assert torch.equal(rows[0][i][~where[i]], rows[1][i][~where[i]])
    # queries: the channel, and its pair's other one where it turns
    at = torch.zeros(T, H, d, device="cuda", dtype=torch.bool)
    at[3, 1, 100] = at[0, 0, 2] = at[0, 0, 18] = True
    assert not out[at].isfinite().any() and torch.equal(out[~at], clean[~at])
    assert q8.q8_device_error() == 0


def test_append_with_no_angle(q8):
    T, Hkv, d = 3, 2, 64
    _, k, v, (_, kw) = fused_rows(T, 1, Hkv, d, BF16, seed=2)
    inv = torch.ones(16, device="cuda", dtype=torch.float64)
    inv[9] = math.inf
    table = q8.q8_rope_table(i32([1, 2, 3]), inv)
    cache = torch.zeros(q8.q8_kv4_cache_shape(1, 32, Hkv, d), device="cuda", dtype=torch.uint8)
    q8.q8_kv4_append(k, v, cache, i32([0, 1, 2]), table=table, k_weight=kw)
    gk, gv = q8.q8_kv4_gather(cache, i32([[0]]), i32([0, T]), T)
    assert not gk[..., :32].isfinite().any() and gk[..., 32:].isfinite().all() and gv.isfinite().all()


def test_append_in_place_repeated_and_strided(q8):
    T, H, Hkv, d, page = 9, 4, 2, 128, 32
    q, k, v, (qw, kw) = fused_rows(T, H, Hkv, d, BF16, seed=5)
    table, slots = table_of(T, 128), list(range(5, 5 + T))
    shape = q8.q8_kv4_cache_shape(2, page, Hkv, d)
    want_c = torch.zeros(shape, device="cuda", dtype=torch.uint8)
    want = q8.q8_kv4_append(k, v, want_c, i32(slots), table=table, q=q, q_weight=qw, k_weight=kw)
    # queries in place, pages apart from one another, one of several layers' caches
    wide = torch.full((2, 3, *shape[1:]), 77, device="cuda", dtype=torch.uint8)
    q2 = q.clone().as_strided(q.shape, (H * d, d, 1)) if q.is_contiguous() else q.contiguous()
    got_c = wide[:, 1]
    got = q8.q8_kv4_append(k, v, got_c, i32(slots), table=table, q=q2, q_weight=qw, k_weight=kw, q_out=q2)
    assert got is q2 and torch.equal(got, want)
    kept, ref = K.unpack(got_c.reshape(-1, 36 * d)), K.unpack(want_c.reshape(-1, 36 * d))
    for x, y in zip(kept, ref):
        assert torch.equal(x.view(2, Hkv, 32, -1)[0, :, 5:14], y.view(2, Hkv, 32, -1)[0, :, 5:14])
    assert bool((wide[:, 0] == 77).all()) and bool((wide[:, 2] == 77).all())
    # one token's rows for all
    one = (k[:1].expand(T, -1, -1), v[:1].expand(T, -1, -1))
    a, b = torch.zeros_like(want_c), torch.zeros_like(want_c)
    q8.q8_kv4_append(*one, a, i32(slots), k_weight=kw)
    q8.q8_kv4_append(*(x.contiguous() for x in one), b, i32(slots), k_weight=kw)
    assert torch.equal(a, b)


def test_append_skips_slots_behind_the_cache(q8):
    T, Hkv, d, page = 4, 2, 64, 32
    _, k, v, _ = fused_rows(T, 1, Hkv, d, BF16, seed=5)
    store = torch.full((4, *q8.q8_kv4_cache_shape(1, page, Hkv, d)[1:]), 9, device="cuda", dtype=torch.uint8)
    cache, before = store[:2], store[:2].clone()
    slots = [64, 7, 2 ** 31 - 1, -2 ** 31]
    q8.q8_kv4_append(k, v, cache, i32(slots))
    check_cache(cache, before, slots, k, v, None, None, False, page)
    assert bool((store[2:] == 9).all())
    assert q8.q8_device_error() == 1 << 10


# ---- a cache with everything that a call must not use --------------------------------------------
def make(lens, page, Hkv, d, seed=0, extra=3, hot=None):
    """cache, block table, and each request's keys, values and scales [n, Hkv, ..]; NaN scales in rows
    behind the lengths and in pages of nobody, table entries of unneeded pages far outside."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    n = pages * Hkv * (page // 32)
    codes = [torch.randint(1, 16, (n, 32, d), generator=g, device="cuda", dtype=I32) for _ in range(2)]
    scales = [(torch.rand(n, 32, d // 32, generator=g, device="cuda") * 0.5 + 0.05).to(BF16) for _ in range(2)]
    if hot is not None:  # a few loud keys
        scales[0][torch.rand(n, 32, generator=g, device="cuda") < 0.02] *= hot
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(need + [1]) + 1
    bt = torch.full((len(lens), width), 2 ** 30, dtype=I32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    at, rows = 0, []
    for b, (m, c) in enumerate(zip(lens, need)):
        mine = perm[at:at + c]
        at += c
        bt[b, :c] = torch.tensor(mine, dtype=I32)
        t = torch.arange(m)
        pg = torch.tensor(mine, dtype=torch.int64)[t // page] if c else torch.zeros(0, dtype=torch.int64)
        used[pg, t % page] = True
        rows.append(((pg[:, None] * Hkv + torch.arange(Hkv)) * (page // 32) + (t % page // 32)[:, None], t % 32))
    free = ~used.view(pages, 1, page // 32, 32).expand(pages, Hkv, -1, -1).reshape(n, 32).cuda()
    for s in scales:
        s.view(torch.int16)[free] = NAN16
    cache = K.pack(*codes, *scales).view(pages, Hkv, page // 32, 36 * d).cuda()
    kv = [K.values(c, s) for c, s in zip(codes, scales)]
    out = []
    for r, t in rows:
        r, t = r.cuda(), t.cuda()[:, None]
        out.append(tuple(x[r, t] for x in (*kv, *scales)))
    return cache, bt.cuda(), out


# ---- gather ------------------------------------------------------------------------------------
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("lens,page,Hkv,d", [
    ([1], 32, 1, 64), ([33, 0, 64, 31, 1], 32, 3, 128), ([0, 0], 64, 2, 64), ([130, 7, 96], 96, 5, 256), ([1000], 64, 8, 128),
    ([5, 250, 64, 65, 63, 0, 300], 256, 2, 64)])
def test_gather(q8, lens, page, Hkv, d, out_dtype):
    cache, bt, kv = make(lens, page, Hkv, d)
    cu = cum(lens)
    T = cu[-1] + 3  # rows behind the last sequence stay
    out = [torch.full((T, Hkv, d), 5.0, device="cuda", dtype=out_dtype) for _ in range(2)]
    got = q8.q8_kv4_gather(cache, bt, i32(cu), T, out_dtype=out_dtype, k=out[0], v=out[1])
    assert q8.q8_device_error() == 0
    for i in range(2):
        want = torch.cat([x[i] for x in kv] + [torch.full((3, Hkv, d), 5.0, device="cuda")])
        assert torch.equal(got[i], want.to(out_dtype))
    # parts of them
    first = [n // 3 for n in lens]
    part = [n - f for n, f in zip(lens, first)]
    got = q8.q8_kv4_gather(cache, bt, i32(cum(part)), sum(part), first=i32(first), out_dtype=out_dtype)
    for i in range(2):
        assert torch.equal(got[i], torch.cat([x[i][f:] for x, f in zip(kv, first)]).to(out_dtype))
    assert q8.q8_device_error() == 0


def test_gather_leaves_what_is_outside(q8):
    cache, bt, kv = make([40, 40], 32, 2, 64)
    bt[0, 1] = cache.shape[0]      # a page behind the cache
    bt[1, 0] = -1
    out = [torch.full((80, 2, 64), 3.0, device="cuda", dtype=F32) for _ in range(2)]
    q8.q8_kv4_gather(cache, bt, i32([0, 40, 80]), 80, out_dtype=F32, k=out[0], v=out[1])
    assert q8.q8_device_error() == 1 << 10
    for i in range(2):
        assert torch.equal(out[i][:32], kv[0][i][:32]) and torch.equal(out[i][72:], kv[1][i][32:])
        assert bool((out[i][32:72] == 3.0).all())
    # tokens in front of the first and behind the table's last
    q8.q8_kv4_gather(cache, bt, i32([0, 8, 16]), 16, first=i32([-8, 32 * bt.shape[1] - 1]))
    assert q8.q8_device_error() == 1 << 10


# ---- attention ---------------------------------------------------------------------------------
def queries(n, H, d, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    return (torch.randn(n, H, d, generator=g, device="cuda") * size).to(BF16)


def expected(q, kv, cu, scale):
    o = torch.full(q.shape, math.nan, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    for (k, v, ks, vs), a, b in zip(kv, cu, cu[1:]):
        seen = torch.ones(b - a, k.shape[0], dtype=torch.bool, device="cuda").tril(k.shape[0] - (b - a))
        o[a:b], tol[a:b] = K.attention(q[a:b], k, v, ks, vs, seen, scale)
    return o, tol


def run(q8, lens, news, page, H, Hkv, d, seed=0, scale=None, size=1.0, hot=None, **kw):
    cache, bt, kv = make(lens, page, Hkv, d, seed, hot=hot)
    cu = cum(news) if news is not None else list(range(len(lens) + 1))
    q = queries(cu[-1], H, d, seed, size)
    o = q8.q8_kv4_attention(q, cache, bt, i32(lens), cu_q=None if news is None else i32(cu), scale=scale, **kw)
    assert q8.q8_device_error() == 0
    R.assert_within(o, *expected(q, kv, cu, d ** -0.5 if scale is None else scale), "attention")
    return q, cache, bt, o


HEADS = [(32, 8, 128), (4, 4, 64), (16, 4, 256), (9, 3, 128), (8, 1, 64), (5, 1, 256), (24, 2, 128), (40, 1, 64), (128, 1, 256)]


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens,page", [([1], 32), ([31, 32, 33], 32), ([1000], 64), ([0, 5, 0, 700, 64, 65], 96)])
def test_one_query_each(q8, H, Hkv, d, lens, page):
    run(q8, lens, None, page, H, Hkv, d, seed=len(lens))


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens,page", [([1], 32), ([0, 33, 500, 32], 64), ([2000], 32)])
def test_wide_block_tables(q8, H, Hkv, d, lens, page):
    """Tables that could name far more keys than there are: the work list instead of clusters."""
    cache, bt, kv = make(lens, page, Hkv, d, seed=5)
    wide = torch.full((len(lens), 5000), -7, device="cuda", dtype=I32)
    wide[:, :bt.shape[1]] = bt
    q = queries(len(lens), H, d)
    want = expected(q, kv, list(range(len(lens) + 1)), d ** -0.5)
    for table in (bt, wide):
        R.assert_within(q8.q8_kv4_attention(q, cache, table, i32(lens)), *want, "attention")
    assert q8.q8_kv4_attention_workspace_size(len(lens), 5000, page, H, Hkv, d) > 0
    if H // Hkv <= 8:
        assert q8.q8_kv4_attention_workspace_size(1, 4, 32, H, Hkv, d) == 0
    assert q8.q8_device_error() == 0


def test_workspace_of_the_caller(q8):
    lens, H, Hkv, d = [3000, 70], 8, 2, 128
    cache, bt, kv = make(lens, 64, Hkv, d)
    q = queries(2, H, d)
    wide = torch.cat((bt, torch.full((2, 300), -1, device="cuda", dtype=I32)), 1).contiguous()
    need = q8.q8_kv4_attention_workspace_size(2, wide.shape[1], 64, H, Hkv, d)
    for fill in (0, 255):  # whatever an earlier call has left there
        ws = torch.full((need,), fill, device="cuda", dtype=torch.uint8)
        o = q8.q8_kv4_attention(q, cache, wide, i32(lens), workspace=ws)
        R.assert_within(o, *expected(q, kv, [0, 1, 2], d ** -0.5))
    with pytest.raises(q8.Q8Error, match="NOMEM"):
        q8.q8_kv4_attention(q, cache, wide, i32(lens), workspace=ws[:need - 16])
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens,news,page", [
    ([7], [7], 32), ([100, 33, 64, 1, 40], [5, 1, 0, 1, 40], 32), ([700, 3], [2, 6], 64), ([0, 130], [3, 17], 128), ([300], [150], 256)])
def test_several_queries(q8, H, Hkv, d, lens, news, page):
    """Drafted tokens; more queries than keys, whose first see none and are 0; requests without a query."""
    run(q8, lens, news, page, H, Hkv, d, seed=len(lens))


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("odd", [math.nan, math.inf])
def test_unseen_tokens_that_are_not_finite(q8, H, Hkv, d, odd):
    """A drafted token's key or value that is not finite stays out of the queries in front of it; what
    sees it is NaN in all its channels."""
    lens, news, page = [70, 33, 5, 64], [6, 4, 5, 1], 32
    cache, bt, kv = make(lens, page, Hkv, d)
    cu = cum(news)
    q = queries(cu[-1], H, d)
    o, tol = expected(q, kv, cu, d ** -0.5)
    bad, lost = (torch.zeros(q.shape, dtype=torch.bool, device="cuda") for _ in range(2))
    tiles = cache.view(cache.shape[0], Hkv, page // 32, 36 * d).clone()
    scales = [tiles[..., at:at + 2 * d].view(BF16).view(cache.shape[0], Hkv, page // 32, d // 32, 32) for at in (16 * d, 34 * d)]
    for b, pos, h, blk, kind in ((0, 66, 0, d // 32 - 1, 1), (0, 68, Hkv - 1, 0, 0), (1, 32, Hkv - 1, 1, 1), (1, 31, 0, 0, 1), (2, 3, 0, 1, 1)):
        scales[kind][int(bt[b, pos // page]), h, 0, blk, pos % page] = odd
        first = max(0, pos - (lens[b] - news[b]))  # the first query that sees it
        heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
        bad[cu[b] + first:cu[b + 1], heads] = True
        if kind == 1 or math.isnan(odd):  # infinity times a negative sum is the score of a key that counts for nothing
            lost[cu[b] + first:cu[b + 1], heads] = True
    got = q8.q8_kv4_attention(q, tiles, bt, i32(lens), cu_q=i32(cu))
    assert q8.q8_device_error() == 0
    assert got[lost].isnan().all()
    R.assert_within(got[~bad], o[~bad], tol[~bad], "queries that do not see it")


@pytest.mark.parametrize("H,Hkv,d,news", [(32, 8, 128, None), (16, 16, 64, None), (16, 4, 256, None), (16, 2, 128, 3), (8, 2, 64, 5)])
def test_long_and_many(q8, H, Hkv, d, news):
    """Runs of the work list that begin and end anywhere: one long request, and many of all lengths."""
    run(q8, [20000], None if news is None else [news], 64, H, Hkv, d, seed=3, hot=8.0)
    lens = [(37 * i * i) % 900 for i in range(70)]
    run(q8, lens, None if news is None else [i % (news + 1) for i in range(70)], 32, H, Hkv, d, seed=4, hot=8.0)


def test_more_requests_than_threads(q8):
    lens = [(7 * i) % 41 for i in range(1100)]
    run(q8, lens, None, 32, 2, 1, 64, seed=9)
    run(q8, lens, [min(n, i % 3) for i, n in enumerate(lens)], 32, 2, 1, 64, seed=9)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scale_and_loud_scores(q8, d):
    """Scores that grow along the keys, large and tiny queries, a scale of the caller's."""
    run(q8, [500, 90], None, 64, 8, 2, d, seed=1, scale=0.3, hot=30.0)
    run(q8, [500, 90], [4, 2], 64, 8, 2, d, seed=1, size=20.0)
    run(q8, [500, 90], None, 64, 8, 2, d, seed=1, size=1e-30)
    run(q8, [64], None, 64, 8, 2, d, seed=1, size=1e12, scale=1e-13)


def test_rows_outside_sequences_stay(q8):
    cache, bt, kv = make([50, 20, 10], 32, 2, 128)
    q = queries(12, 4, 128)
    o = torch.full(q.shape, 7.0, device="cuda", dtype=BF16)
    # the second sequence is malformed (behind Tq), the third fine, the rows in front of the first nobody's
    q8.q8_kv4_attention(q, cache, bt, i32([50, 20, 10]), cu_q=i32([1, 4, 13, 6]), o=o)
    assert q8.q8_device_error() == 1 << 10
    ref, tol = expected(q, kv[:1], [1, 4], 128 ** -0.5)
    R.assert_within(o[1:4], ref[1:4], tol[1:4])
    assert bool((o[0] == 7.0).all()) and bool((o[4:] == 7.0).all())
    o.fill_(7.0)
    q8.q8_kv4_attention(q, cache, bt, i32([50, 20, 10]), cu_q=i32([1, 4, 4, 6]), o=o)
    assert q8.q8_device_error() == 0
    ref, tol = expected(q, [kv[0], kv[1], kv[2]], [1, 4, 4, 6], 128 ** -0.5)
    R.assert_within(o[1:6], ref[1:6], tol[1:6])
    assert bool((o[0] == 7.0).all()) and bool((o[6:] == 7.0).all())


def test_pages_and_lengths_outside(q8):
    cache, bt, kv = make([100, 64, 32], 32, 2, 128, extra=4)
    q = queries(3, 4, 128)
    bt[0, 1] = cache.shape[0]
    bt[1, 0] = -5
    o = q8.q8_kv4_attention(q, cache, bt, i32([100, 64, -3]))
    assert q8.q8_device_error() == 1 << 10
    keep = torch.arange(100, device="cuda")
    a = [x[(keep < 32) | (keep >= 64)] for x in kv[0]]
    b = [x[32:] for x in kv[1]]
    c = [x[:0] for x in kv[2]]
    R.assert_within(o, *expected(q, [a, b, c], [0, 1, 2, 3], 128 ** -0.5))
    # a length behind the table's last page is that page's end
    bt2 = bt[2:, :1].contiguous()
    o = q8.q8_kv4_attention(q[2:], cache, bt2, i32([2 ** 31 - 1]))
    assert q8.q8_device_error() == 1 << 10
    R.assert_within(o, *expected(q[2:], [kv[2]], [0, 1], 128 ** -0.5))


def test_strided_queries_outputs_and_pages(q8):
    lens, H, Hkv, d = [70, 200, 3], 8, 2, 128
    cache, bt, kv = make(lens, 64, Hkv, d)
    wide = torch.full((cache.shape[0], 2, *cache.shape[1:]), 255, device="cuda", dtype=torch.uint8)
    wide[:, 1] = cache
    q = queries(3, H, d)
    rows = torch.zeros(3, H + 4, 2 * d, device="cuda", dtype=BF16)
    qs = rows[:, 2:2 + H, d:]
    qs.copy_(q)
    heads_first = torch.zeros(H, 3, d, device="cuda", dtype=BF16)
    want = q8.q8_kv4_attention(q, cache, bt, i32(lens))
    got = q8.q8_kv4_attention(qs, wide[:, 1], bt, i32(lens), o=heads_first.transpose(0, 1))
    assert torch.equal(got, want)
    R.assert_within(want, *expected(q, kv, [0, 1, 2, 3], d ** -0.5))


def test_pages_and_rows_far_apart(q8):
    """Byte offsets of pages, and element offsets of rows, that pass 32 bits."""
    lens, H, Hkv, d, page = [70, 40], 8, 2, 64, 32
    cache, bt, kv = make(lens, page, Hkv, d, extra=0)
    pages, size, far = cache.shape[0], Hkv * 36 * d, 5 << 28  # 1.25 GiB between pages
    store = torch.empty((pages - 1) * far + size, device="cuda", dtype=torch.uint8)
    wide = store.as_strided(cache.shape, (far, 36 * d, 36 * d, 1))
    wide.copy_(cache)
    assert (pages - 1) * far > 1 << 32
    q = queries(2, H, d)
    rows = torch.empty((1 << 32) + H * d, device="cuda", dtype=BF16).as_strided((2, H, d), (1 << 32, d, 1))
    rows.copy_(q)
    for table in (bt, widened(bt)):
        R.assert_within(q8.q8_kv4_attention(rows, wide, table, i32(lens)), *expected(q, kv, [0, 1, 2], d ** -0.5))
    out = torch.zeros((1 << 32) + H * d, device="cuda", dtype=BF16).as_strided((2, H, d), (1 << 32, d, 1))
    R.assert_within(q8.q8_kv4_attention(q, cache, bt, i32(lens), o=out), *expected(q, kv, [0, 1, 2], d ** -0.5))
    k, v = q8.q8_kv4_gather(wide, bt, i32([0, 70, 110]), 110, out_dtype=F32)
    assert torch.equal(k, torch.cat([x[0] for x in kv])) and torch.equal(v, torch.cat([x[1] for x in kv]))
    slot = int(bt[1, 1]) * page + 9
    x = torch.randn(1, Hkv, d, device="cuda")
    q8.q8_kv4_append(x, x, wide, i32([slot]))
    q8.q8_kv4_append(x, x, cache, i32([slot]))
    assert torch.equal(wide, cache) and q8.q8_device_error() == 0


def test_nothing_to_do(q8):
    cache, bt, _ = make([5], 32, 2, 64)
    q = queries(0, 4, 64)
    assert q8.q8_kv4_attention(q, cache, bt[:0], i32([])).shape == (0, 4, 64)
    assert q8.q8_kv4_attention(q, cache, bt, i32([5]), cu_q=i32([0, 0])).shape == (0, 4, 64)
    # no page at all: nothing is seen
    o = q8.q8_kv4_attention(queries(1, 4, 64), cache[:0], bt[:, :0], i32([0]))
    assert torch.equal(o, torch.zeros_like(o)) and q8.q8_device_error() == 0
    k, v = q8.q8_kv4_gather(cache, bt, i32([0, 0]), 0)
    assert k.shape == v.shape == (0, 2, 64)
    e = torch.zeros(0, 2, 64, device="cuda", dtype=BF16)
    assert q8.q8_kv4_append(e, e, cache, i32([]), q=e).shape == (0, 2, 64)
    assert q8.q8_rope_table(i32([]), torch.ones(8, device="cuda", dtype=torch.float64)).shape == (0, 2, 8)
    assert q8.q8_device_error() == 0


def test_the_same_every_time(q8):
    """Sums are taken in an order fixed by the lengths."""
    cache, bt, _ = make([3000, 50, 700], 64, 4, 128, seed=2)
    q = queries(3, 16, 128)
    for table in (bt, widened(bt)):
        first = q8.q8_kv4_attention(q, cache, table, i32([3000, 50, 700]))
        for _ in range(20):
            assert torch.equal(q8.q8_kv4_attention(q, cache, table, i32([3000, 50, 700])), first)


# ---- as they are used --------------------------------------------------------------------------
def test_a_decode_loop_and_its_graph(q8):
    """Prompts appended in one call, then tokens one by one: every step's attention against the cache
    as it stands; the same steps captured once and replayed with lengths that grow."""
    H, Hkv, d, page, lens = 8, 2, 128, 32, [45, 3, 31]
    B, steps = len(lens), 4
    inv = 1e6 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    width = 3
    bt = i32([[7, 0, 5], [2, 9, 4], [8, 3, 6]])
    at = lambda b, t: int(bt[b, t // page]) * page + t % page  # noqa: E731

    def step_inputs(s):
        q, k, v, w = fused_rows(B, H, Hkv, d, BF16, seed=50 + s)
        return q, k, v, i32([n + s for n in lens]), i32([at(b, n + s) for b, n in enumerate(lens)]), i32([n + s + 1 for n in lens])

    def fresh():
        cache = torch.zeros(q8.q8_kv4_cache_shape(10, page, Hkv, d), device="cuda", dtype=torch.uint8)
        T = sum(lens)
        _, k, v, (_, kw) = fused_rows(T, H, Hkv, d, BF16, seed=1)
        pos = i32([t for n in lens for t in range(n)])
        slots = i32([at(b, t) for b, n in enumerate(lens) for t in range(n)])
        q8.q8_kv4_append(k, v, cache, slots, table=q8.q8_rope_table(pos, inv), k_weight=kw)
        return cache, kw

    cache, kw = fresh()
    eager = []
    for s in range(steps):
        q, k, v, pos, slots, n = step_inputs(s)
        qr = q8.q8_kv4_append(k, v, cache, slots, table=q8.q8_rope_table(pos, inv), q=q, q_weight=kw, k_weight=kw)
        o = q8.q8_kv4_attention(qr, cache, bt, n)
        total = int(n.sum())
        kk, vv = q8.q8_kv4_gather(cache, bt, i32(cum(n.tolist())), total, out_dtype=F32)
        kv, a = [], 0
        for b, m in enumerate(n.tolist()):
            t = torch.arange(m)
            rows = torch.stack([((bt[b, t // page].cpu().long() * Hkv + h) + 0 * t) for h in range(Hkv)], 1)
            _, _, ks, vs = K.unpack(cache.reshape(-1, 36 * d))
            kv.append((kk[a:a + m], vv[a:a + m], ks[rows, t[:, None] % 32].cuda(), vs[rows, t[:, None] % 32].cuda()))
            a += m
        R.assert_within(o, *expected(qr, kv, list(range(B + 1)), d ** -0.5), f"step {s}")
        # the same as whole-prompt attention over the keys and values read back in bfloat16, within both's rounding
        kb, vb = q8.q8_kv4_gather(cache, bt, i32(cum(n.tolist())), total)
        ob = q8.q8_prompt_attention(qr, kb, vb, i32(list(range(B + 1))), i32(cum(n.tolist())))
        assert float((ob.float() - o.float()).norm() / o.float().norm()) < 0.02
        eager.append((qr.clone(), o.clone(), cache.clone()))
    assert q8.q8_device_error() == 0

    cache2, _ = fresh()
    q, k, v, pos, slots, n = (x.clone() for x in step_inputs(0))

    def step():
        qr = q8.q8_kv4_append(k, v, cache2, slots, table=q8.q8_rope_table(pos, inv), q=q, q_weight=kw, k_weight=kw)
        return qr, q8.q8_kv4_attention(qr, cache2, bt, n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for s in range(steps):
        for dst, src in zip((q, k, v, pos, slots, n), step_inputs(s)):
            dst.copy_(src)
        graph.replay()
        assert torch.equal(outs[0], eager[s][0]) and torch.equal(outs[1], eager[s][1]) and torch.equal(cache2, eager[s][2])
    assert width == bt.shape[1] and q8.q8_device_error() == 0


def widened(bt, width=3000):
    """The block table with room for many more pages: calls go through the work list."""
    return torch.cat((bt, torch.full((bt.shape[0], width - bt.shape[1]), 2 ** 30, device="cuda", dtype=I32)), 1).contiguous()


@pytest.mark.parametrize("news", [None, [1, 3, 0, 2]])
def test_a_graph_of_the_work_list(q8, news):
    """Captured once, replayed with other lengths, queries and pages, among other work on the stream."""
    H, Hkv, d, page, B = 16, 4, 128, 64, 4
    sets = []
    for i, lens in enumerate(([5000, 3, 700, 64], [1, 4000, 33, 2], [600, 610, 620, 6300])):
        cache, bt, kv = make(lens, page, Hkv, d, seed=i, extra=3)
        sets.append((lens, cache, widened(bt, 200), kv, queries(B if news is None else sum(news), H, d, seed=i)))
    pages = max(s[1].shape[0] for s in sets)
    cache = torch.zeros((pages, *sets[0][1].shape[1:]), device="cuda", dtype=torch.uint8)
    bt, q, n = torch.empty_like(sets[0][2]), torch.empty_like(sets[0][4]), i32([0] * B)
    cu = None if news is None else i32(cum(news))

    def load(s):
        cache[:s[1].shape[0]].copy_(s[1])
        bt.copy_(s[2])
        q.copy_(s[4])
        n.copy_(i32(s[0]))

    load(sets[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q8.q8_kv4_attention(q, cache, bt, n, cu_q=cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = q8.q8_kv4_attention(q, cache, bt, n, cu_q=cu)
        twice = o * 2
    for s in sets + sets[:1]:
        load(s)
        graph.replay()
        want = expected(s[4], s[3], cum(news) if news else list(range(B + 1)), d ** -0.5)
        R.assert_within(o, *want, "replay")
        assert torch.equal(twice, o * 2)
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("B,wide", [(1, False), (1, True), (4, False), (4, True)])
def test_layers_one_behind_the_other(q8, B, wide):
    """Kernels of a step may start while the ones in front of them end: layers of projections, rotations,
    cache and attention without a pause, waited for one by one, and captured, give the same bits."""
    H, Hkv, d, page, layers, n = 8, 2, 128, 32, 6, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    inv = 1e6 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    kv_len, pos = i32([n + 1] * B), i32([n] * B)
    ws = [[q8.q8_quantize_weights(torch.randn(rows, H * d, generator=g, device="cuda") * 0.03) for rows in ((H + 2 * Hkv) * d, H * d)]
          for _ in range(layers)]
    x0 = torch.randn(B, H * d, generator=g, device="cuda").to(BF16)
    kw = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    made = [make([n] * B, page, Hkv, d, seed=i, extra=0)[:2] for i in range(layers)]
    start = [cache for cache, _ in made]
    tables = [(widened(bt) if wide else bt, bt[:, n // page] * page + n % page) for _, bt in made]

    def go(caches, wait):
        x, out = x0, []
        for (wqkv, wo), cache, (bt, place) in zip(ws, caches, tables):
            table = q8.q8_rope_table(pos, inv)
            wait()
            y = q8.q8_linear_ex(x, *wqkv).view(B, H + 2 * Hkv, d)
            wait()
            q = q8.q8_kv4_append(y[:, H:H + Hkv], y[:, H + Hkv:], cache, place, table=table, q=y[:, :H], q_weight=kw, k_weight=kw)
            wait()
            o = q8.q8_kv4_attention(q, cache, bt, kv_len)
            wait()
            x = q8.q8_linear_ex(o.view(B, H * d), *wo).to(BF16)
            wait()
            out += [q, o, x]
        return out

    slow = [c.clone() for c in start]
    want = go(slow, torch.cuda.synchronize)
    assert all(x.isfinite().all() for x in want)
    for _ in range(5):
        fast = [c.clone() for c in start]
        assert all(torch.equal(a, b) for a, b in zip(go(fast, lambda: None) + fast, want + slow))
    fast = [c.clone() for c in start]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go(fast, lambda: None)
    for _ in range(5):
        for c, s in zip(fast, start):
            c.copy_(s)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got + fast, want + slow))
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("wide", [False, True])
def test_captured_behind_copies_and_joins(q8, wide):
    """Calls that follow a fill, a copy, a copy on another stream or two streams at once, eager and captured."""
    lens, page, H, Hkv, d = [40, 64], 32, 8, 2, 128
    source, bt, kv = make(lens, page, Hkv, d)
    bt = widened(bt) if wide else bt
    T, n, cu = 2, i32([41, 65]), i32([0, 41, 106])
    q, k, v, (qw, kw) = fused_rows(T, H, Hkv, d, BF16, seed=9)
    used = {int(p) for p in bt[:, :2].flatten().tolist() if 0 <= p < source.shape[0]}
    free = [p for p in range(source.shape[0]) if p not in used]
    bt[1, 2] = free[0]
    slots = i32([int(bt[0, 1]) * page + 8, free[0] * page])
    pos, inv = i32([40, 64]), 1e4 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) / 64)
    host = source.cpu().pin_memory()
    cache, rows = torch.empty_like(source), [torch.empty(106, Hkv, d, device="cuda", dtype=BF16) for _ in range(2)]
    side = torch.cuda.Stream()

    def go():
        main = torch.cuda.current_stream()
        cache.copy_(host, non_blocking=True)  # a copy in front of the table
        table = q8.q8_rope_table(pos, inv)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            qs = q.clone()
            cache[:, :, :, :16].copy_(source[:, :, :, :16])
        main.wait_stream(side)  # two streams in front of the append
        qr = q8.q8_kv4_append(k, v, cache, slots, table=table, q=qs, q_weight=qw, k_weight=kw)
        for r in rows:
            r.zero_()  # a fill in front of the gather
        q8.q8_kv4_gather(cache, bt, cu, 106, k=rows[0], v=rows[1])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            other = q8.q8_kv4_attention(qr, cache, bt, n)
        o = q8.q8_kv4_attention(qr, cache, bt, n)
        main.wait_stream(side)
        return [qr, o, other, *rows, cache]

    eager = [x.clone() for x in go()]
    assert all(x.isfinite().all() for x in eager[:5]) and torch.equal(eager[1], eager[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
    assert q8.q8_device_error() == 0


def test_streams_overlap(q8):
    """Two calls on two streams at once, each with a workspace of its own."""
    sets = [make([2000 + 100 * i, 50], 64, 4, 128, seed=i) for i in range(2)]
    sets = [(c, widened(bt), kv) for c, bt, kv in sets]
    qs = [queries(2, 16, 128, seed=i) for i in range(2)]
    ns = [i32([2000 + 100 * i, 50]) for i in range(2)]
    want = [q8.q8_kv4_attention(q, c, bt, n) for q, (c, bt, _), n in zip(qs, sets, ns)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [q8.q8_kv4_attention(q, c, bt, n, stream=s) for q, (c, bt, _), n, s in zip(qs, sets, ns, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert q8.q8_device_error() == 0
