"""The 4-bit cache: every variant that the host's rules choose by size, type and pairing, with the rule
beside it, so that a case that no longer reaches its variant says so."""
import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402
from tests import kv4_ref as K  # noqa: E402
from tests.test_gpu_kv4 import (BF16, F32, check_q, cum, expected, fused_rows, i32, make, q8, queries,  # noqa: E402, F401
                                table_of, widened)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def up(a, b):
    return -(-a // b)


# ---- append ------------------------------------------------------------------------------------
def append_variant(T, H, Hkv, d):
    """"tiles", or how many rounds of heads a warp takes."""
    if T >= 32 and up(T, 32) * up(Hkv, 2) >= 2 * sms():
        return "tiles"
    teams = 256 // d
    return 2 if T * (up(H, 2 * teams) + 2 * up(Hkv, teams)) >= 32 * sms() else 1


def check_bytes(cache, before, slots, k, v, kw, table, interleaved, page, eps=1e-6):
    """The bytes of the cache: codes and scales bit for bit, a scale bfloat16(fl(fl(amax r) fl(1/7))) with r = 1
    where there is no norm (with a norm the order of its sum is the kernel's: within a step of binary64's r);
    everything else as it was."""
    pages, Hkv, tiles, _ = cache.shape
    d = k.shape[2]
    put = [t for t, s in enumerate(slots) if 0 <= s < pages * page]
    assert put
    seventh = torch.tensor(1.0, dtype=F32) / 7.0
    kc, ktop = K.quantised(K.turned(k.cpu(), None if kw is None else kw.cpu(), None if table is None else table.cpu(), interleaved))
    vc, vtop = K.quantised(v.cpu().float())
    if kw is not None:
        ktop = (ktop.double() / (k.cpu().double().square().mean(-1, keepdim=True) + eps).sqrt()).float()
    want, got = [x.clone() for x in K.unpack(before.reshape(-1, 36 * d))], K.unpack(cache.reshape(-1, 36 * d))
    where = torch.tensor([slots[t] for t in put])
    rows = (where // page * Hkv)[:, None] * tiles + torch.arange(Hkv) * tiles + (where % page // 32)[:, None]
    for x, y in zip(want, (kc, vc, (ktop * seventh).to(BF16), (vtop * seventh).to(BF16))):
        x[rows, (where % 32)[:, None]] = y[torch.tensor(put)].to(x.dtype)
    for i, name in enumerate(("key codes", "value codes", "key scales", "value scales")):
        a, b = (x[i] if i < 2 else x[i].view(torch.int16).int() for x in (got, want))
        far = int((a - b).abs().max())
        assert far <= (1 if i == 2 and kw is not None else 0), (name, far, int((a != b).sum()))


def check_append(q8, slots, H, Hkv, d, rot, page, pages, norm, dtype, interleaved, error=0):  # noqa: F811
    T = len(slots)
    q, k, v, (qw, kw) = fused_rows(T, H, Hkv, d, dtype, seed=T + d + Hkv)
    qw, kw = (qw if H else None, kw) if norm else (None, None)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, q8.q8_kv4_cache_shape(pages, page, Hkv, d), generator=g, device="cuda", dtype=torch.uint8)
    before, table = cache.clone(), table_of(T, rot)
    out = q8.q8_kv4_append(k, v, cache, i32(slots), table=table, q=q if H else None, q_weight=qw, k_weight=kw,
                           interleaved=interleaved)
    assert q8.q8_device_error() == error
    check_bytes(cache, before, slots, k, v, kw, table, interleaved, page)
    if H:
        check_q(out, q, qw, table, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,Hkv,d,rot,norm", [
    (1, 32, 8, 128, 128, True), (1, 1, 1, 64, 64, False), (1, 16, 4, 256, 64, True), (1, 0, 3, 128, 0, True), (1, 5, 5, 64, 16, True),
    (2, 32, 8, 128, 64, False), (2, 5, 5, 64, 32, True), (2, 3, 1, 256, 256, True)])
def test_append_of_one_token_and_two(q8, T, H, Hkv, d, rot, norm, dtype, interleaved):  # noqa: F811
    slots = [77, 31][:T]
    check_append(q8, slots, H, Hkv, d, rot, 32, 3, norm, dtype, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,Hkv,d,rot,page,norm", [
    (1000, 16, 4, 256, 64, 96, True), (333, 15, 5, 256, 256, 64, True), (999, 0, 3, 256, 0, 32, False),
    (700, 40, 5, 64, 64, 64, True), (1217, 9, 9, 64, 48, 256, False), (801, 32, 8, 128, 128, 64, True)])
def test_append_by_two_rounds(q8, T, H, Hkv, d, rot, page, norm, dtype, interleaved):  # noqa: F811
    assert append_variant(T, H, Hkv, d) == 2
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].tolist()
    slots[T // 2], slots[T - 1], slots[3] = -1, pages * page, -T
    check_append(q8, slots, H, Hkv, d, rot, page, pages, norm, dtype, interleaved, error=1 << 10)


@pytest.mark.parametrize("dtype,interleaved", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("runs,H,Hkv,d,rot,page,norm", [
    ([(5, 1300)], 4, 16, 128, 128, 64, True), ([(77, 700), (5, 1), (31, 33), (64, 320)], 2, 64, 64, 64, 32, True),
    ([(13, 1000), (200, 31)], 3, 20, 256, 64, 96, True), ([(1, 700)], 0, 31, 128, 96, 256, False)])
def test_append_through_tiles(q8, runs, H, Hkv, d, rot, page, norm, dtype, interleaved):  # noqa: F811
    T = sum(n for _, n in runs)
    assert append_variant(T, H, Hkv, d) == "tiles"
    need = [up(a + n, page) for a, n in runs]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(T)).tolist()
    slots, at = [], 0
    for (a, n), m in zip(runs, need):
        slots += [perm[at + t // page] * page + t % page for t in range(a, a + n)]
        at += m
    check_append(q8, slots, H, Hkv, d, rot, page, pages, norm, dtype, interleaved)
    slots[40:90], slots[T // 2] = [-3] * 50, pages * page
    check_append(q8, slots, H, Hkv, d, rot, page, pages, norm, dtype, interleaved, error=1 << 10)


# ---- gather ------------------------------------------------------------------------------------
def gather_many(T, Hkv):
    """32 rows a warp."""
    return up(T, 32) * Hkv >= 8 * sms()


def check_gather(q8, lens, page, Hkv, d, out_dtype):  # noqa: F811
    cache, bt, kv = make(lens, page, Hkv, d, seed=len(lens))
    cu = cum(lens)
    T = cu[-1] + 3  # rows behind the last sequence stay
    out = [torch.full((T, Hkv, d), 5.0, device="cuda", dtype=out_dtype) for _ in range(2)]
    got = q8.q8_kv4_gather(cache, bt, i32(cu), T, out_dtype=out_dtype, k=out[0], v=out[1])
    for i in range(2):
        want = torch.cat([x[i] for x in kv] + [torch.full((3, Hkv, d), 5.0, device="cuda")])
        assert torch.equal(got[i], want.to(out_dtype))
    first = [n // 3 for n in lens]
    part = [n - f for n, f in zip(lens, first)]
    got = q8.q8_kv4_gather(cache, bt, i32(cum(part)), sum(part), first=i32(first), out_dtype=out_dtype)
    for i in range(2):
        assert torch.equal(got[i], torch.cat([x[i][f:] for x, f in zip(kv, first)]).to(out_dtype))
    assert q8.q8_device_error() == 0
    return cache, bt, kv, cu


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("lens,page,Hkv,d", [
    ([2400, 33, 0, 1950, 31], 64, 16, 64), ([6000, 1, 1300, 63], 32, 8, 128), ([1200, 850, 1000], 96, 20, 256), ([1700], 256, 41, 64)])
def test_gather_of_many_rows(q8, lens, page, Hkv, d, out_dtype):  # noqa: F811
    assert gather_many(sum(n - n // 3 for n in lens), Hkv)
    cache, bt, kv, cu = check_gather(q8, lens, page, Hkv, d, out_dtype)
    # rows of pages and tokens outside the cache stay
    bt = bt.clone()
    bt[0, 1], bt[0, 3] = cache.shape[0], -1
    T = cu[-1]
    out = [torch.full((T, Hkv, d), 5.0, device="cuda", dtype=out_dtype) for _ in range(2)]
    q8.q8_kv4_gather(cache, bt, i32(cu), T, out_dtype=out_dtype, k=out[0], v=out[1])
    assert q8.q8_device_error() == 1 << 10
    for i in range(2):
        want = torch.cat([x[i] for x in kv])
        want[page:2 * page] = 5.0
        want[3 * page:4 * page] = 5.0
        assert torch.equal(out[i], want.to(out_dtype))


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("Hkv,d", [(1, 256), (2, 128), (41, 64)])
@pytest.mark.parametrize("lens", [
    [(7 * i) % 5 for i in range(1100)], [0] * 50 + [100] + [0] * 40 + [1] * 1500 + [0] * 70, [1, 0, 0] * 1000, [0] * 33 + [40] * 40 + [0, 0]])
def test_gather_of_many_requests(q8, lens, Hkv, d, out_dtype):  # noqa: F811
    """More requests than a warp looks at in one step, more than 32 that begin in one warp's rows, empty ones."""
    assert len(lens) > 32 and gather_many(sum(lens), Hkv) == (Hkv == 41)
    check_gather(q8, lens, 32, Hkv, d, out_dtype)


# ---- attention ---------------------------------------------------------------------------------
def check_attention(q8, lens, H, Hkv, d, page, alone, cu=False):  # noqa: F811
    cache, bt, kv = make(lens, page, Hkv, d, seed=H)
    if not alone and not cu:
        bt = widened(bt)
    B = len(lens)
    assert (q8.q8_kv4_attention_workspace_size(B, bt.shape[1], page, H, Hkv, d, one_query=not cu) == 0) == alone
    q = queries(B, H, d)
    o = q8.q8_kv4_attention(q, cache, bt, i32(lens), cu_q=i32(list(range(B + 1))) if cu else None)
    assert q8.q8_device_error() == 0
    R.assert_within(o, *expected(q, kv, list(range(B + 1)), d ** -0.5), "attention")


@pytest.mark.parametrize("alone", [True, False])
@pytest.mark.parametrize("H,Hkv,d", [(32, 2, 64), (9, 1, 64), (33, 3, 64), (16, 16, 64), (16, 1, 128), (33, 3, 128), (7, 1, 128), (8, 1, 256)])
@pytest.mark.parametrize("lens,page", [([1], 32), ([33, 500, 0, 64], 64), ([1411], 32)])
def test_groups_of_any_size(q8, H, Hkv, d, lens, page, alone):  # noqa: F811
    check_attention(q8, lens, H, Hkv, d, page, alone)


@pytest.mark.parametrize("H,Hkv,d", [(8, 8, 64), (32, 8, 128), (16, 8, 256), (128, 8, 128)])
@pytest.mark.parametrize("requests,blocks", [(1, 8), (4, 4), (8, 2), (19, 1)])
def test_clusters_of_each_size(q8, H, Hkv, d, requests, blocks):  # noqa: F811
    items = requests * Hkv
    c = 8
    while c > 1 and 8 * items * c > (6 if c == 8 else 7) * sms():
        c //= 2
    assert c == blocks and items <= sms()
    check_attention(q8, [(997 * (i + 1)) % (1500 * c) for i in range(requests)], H, Hkv, d, 32, True)


@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (8, 8, 64), (16, 4, 256), (32, 2, 64), (24, 2, 128)])
def test_single_queries_named_by_their_rows(q8, H, Hkv, d):  # noqa: F811
    """One query each, given with cu_q as a server with mixed batches does."""
    check_attention(q8, [1, 700, 33, 0, 64, 2000], H, Hkv, d, 64, False, cu=True)
