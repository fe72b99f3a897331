"""Attention over packed prompts (q8_prompt_attention) and behind a shared prefix
(q8_prefix_attention) against their binary64 forms; the tolerance is derived in
tests/attention_ref.py."""
import itertools

import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


def _rand(seed, *shape, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(BF16)


def _cum(n):
    c = [0] + list(itertools.accumulate(n))
    return c, torch.tensor(c, dtype=torch.int32, device="cuda")


def _prompt(q8, nq, nk, H, Hkv, d, seed=0, gain=1.0, **kw):
    (cq, tq), (ck, tk) = _cum(nq), _cum(nk)
    q, k, v = _rand(seed, cq[-1], H, d, gain=gain), _rand(seed + 1, ck[-1], Hkv, d), _rand(seed + 2, ck[-1], Hkv, d)
    o = q8.q8_prompt_attention(q, k, v, tq, None if nk == nq else tk, **kw)
    assert o.dtype == BF16 and o.shape == q.shape
    R.assert_within(o, *R.prompt(q, k, v, cq, ck, kw.get("scale")), f"{nq} {nk} {H}/{Hkv} d={d}")
    assert q8.q8_device_error() == 0
    return q, k, v, tq, tk, o


# ---- packed prompts ------------------------------------------------------------------------
HEADS = [(1, 1, 128), (4, 1, 128), (8, 2, 64), (3, 3, 64), (5, 1, 128), (6, 2, 128), (32, 1, 64)]


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("n", [[1], [2, 1, 3], [127], [128], [129], [64, 65, 63], [0, 1, 0, 130, 0], [257, 300],
                               [1] * 40, [33, 511, 7]])
def test_prompts_of_many_lengths(q8, n, H, Hkv, d):
    _prompt(q8, n, n, H, Hkv, d, seed=sum(n))


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (2, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("nq,nk", [([1], [1000]), ([5, 1], [5, 700]), ([130], [131]), ([3, 200], [900, 201]),
                                   ([1] * 9, [1, 2, 63, 64, 65, 127, 128, 129, 500]), ([64, 17], [640, 1041])])
def test_new_tokens_behind_a_cache(q8, nq, nk, H, Hkv, d):
    _prompt(q8, nq, nk, H, Hkv, d, seed=3)


@pytest.mark.parametrize("nq,nk", [([4], [1]), ([300, 5], [200, 0]), ([10, 140, 1], [0, 10, 0]), ([3], [0])])
def test_queries_without_a_key_get_zero(q8, nq, nk):
    q, k, v, tq, tk, o = _prompt(q8, nq, nk, 8, 2, 128, seed=4)
    at = 0
    for a, b in zip(nq, nk):
        assert (o[at:at + max(0, a - b)] == 0).all()
        at += a


@pytest.mark.parametrize("G,Hkv,d", [(128, 1, 64), (100, 1, 128), (65, 2, 128), (16, 2, 128), (9, 1, 64)])
def test_wide_groups(q8, G, Hkv, d):
    _prompt(q8, [3, 150], [3, 150], G * Hkv, Hkv, d, seed=G)


def test_long_prompt_sampled(q8):
    """9001 tokens: sampled rows against the plain form."""
    n, H, Hkv, d = 9001, 8, 2, 128
    q, k, v = _rand(1, n, H, d), _rand(2, n, Hkv, d), _rand(3, n, Hkv, d)
    o = q8.q8_prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    for t in (0, 1, 127, 128, 4095, 4096, 6000, 8999, 9000):
        ref = R.prompt(q[t:t + 1], k[:t + 1], v[:t + 1], [0, 1], [0, t + 1])
        R.assert_within(o[t:t + 1], *ref, f"row {t}")
    assert q8.q8_device_error() == 0


def test_one_token_behind_a_long_cache(q8):
    for d, H, Hkv in ((128, 8, 2), (64, 4, 4)):
        _prompt(q8, [1], [40001], H, Hkv, d, seed=9)
        _prompt(q8, [1, 7], [30000, 11], H, Hkv, d, seed=9)


@pytest.mark.parametrize("gain", [0.0, 8.0, 40.0])
def test_flat_and_sharp_scores(q8, gain):
    _prompt(q8, [260, 31], [500, 31], 4, 2, 128, seed=5, gain=gain)


def test_maximum_rising_along_the_keys(q8):
    """Keys that grow: most blocks raise the rows' maximum far above the one before."""
    n, H, Hkv, d = 1300, 4, 2, 128
    q, k, v = _rand(1, n, H, d), _rand(2, n, Hkv, d), _rand(3, n, Hkv, d)
    k = (k.float() * (0.5 + torch.arange(n, device="cuda") / 40)[:, None, None]).to(BF16)
    c, t = _cum([n])
    o = q8.q8_prompt_attention(q, k, v, t)
    R.assert_within(o, *R.prompt(q, k, v, c, c), "rising")
    o = q8.q8_prompt_attention(q[-5:], k, v, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), t)
    R.assert_within(o, *R.prompt(q[-5:], k, v, [0, 5], c), "rising, few queries")


def test_own_scale(q8):
    _prompt(q8, [70, 5], [70, 5], 4, 2, 64, seed=6, scale=0.3)
    _prompt(q8, [70], [300], 4, 2, 128, seed=6, scale=0.01)


@pytest.mark.parametrize("d", [64, 128])
def test_layouts(q8, d):
    """Views of a projection's rows; each head's tokens together; a strided o; one key head
    for all (stride 0)."""
    n, H, Hkv = [100, 1, 211], 6, 2
    c, t = _cum(n)
    T = c[-1]
    x = _rand(7, T, (H + 2 * Hkv) * d + 8)
    q = x[:, :H * d].view(T, H, d)
    k, v = (x[:, (H + i * Hkv) * d:(H + (i + 1) * Hkv) * d].view(T, Hkv, d) for i in (0, 1))
    ref = R.prompt(q, k, v, c, c)
    o = q8.q8_prompt_attention(q, k, v, t)
    R.assert_within(o, *ref, "rows of a projection")
    major = lambda y: y.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    om = major(torch.full((T, H, d), NAN, dtype=BF16, device="cuda"))
    got = q8.q8_prompt_attention(major(q), major(k), major(v), t, o=om)
    assert got is om and torch.equal(om, o)
    wide = torch.full((T, H, d + 16), NAN, dtype=BF16, device="cuda")
    q8.q8_prompt_attention(q, k, v, t, o=wide[..., :d])
    assert torch.equal(wide[..., :d], o) and wide[..., d:].isnan().all()
    k1, v1 = k[:, :1].expand(T, Hkv, d), v[:, :1].expand(T, Hkv, d)
    R.assert_within(q8.q8_prompt_attention(q, k1, v1, t), *R.prompt(q, k1, v1, c, c), "one key head repeated")


def test_rows_outside_the_sequences_are_left(q8):
    H, Hkv, d = 4, 2, 128
    q, k, v = _rand(1, 300, H, d), _rand(2, 400, Hkv, d), _rand(3, 400, Hkv, d)
    cq, ck = [10, 150, 150, 260], [30, 170, 200, 390]
    t = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    o = torch.full((300, H, d), NAN, dtype=BF16, device="cuda")
    q8.q8_prompt_attention(q, k, v, t(cq), t(ck), o=o)
    R.assert_within(o, *R.prompt(q, k, v, cq, ck), "gaps")  # NaN outside, as the reference
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("value", [NAN, float("inf")])
@pytest.mark.parametrize("nq,nk", [([100, 90, 70], [100, 90, 70]), ([2, 3, 1], [300, 17, 90]), ([1, 1, 1], [1, 5, 64])])
def test_a_sequence_does_not_reach_its_neighbours(q8, nq, nk, value):
    H, Hkv, d = 4, 2, 128
    (cq, tq), (ck, tk) = _cum(nq), _cum(nk)
    pad = 40  # rows behind the last sequence
    q, k, v = _rand(1, cq[-1] + pad, H, d), _rand(2, ck[-1] + pad, Hkv, d), _rand(3, ck[-1] + pad, Hkv, d)
    ref = R.prompt(q, k, v, cq, ck)
    for x in (q, k, v):
        c = cq if x is q else ck
        x[c[1]:c[2]] = value
        x[c[-1]:] = value
    o = torch.full_like(q, 3.0)
    q8.q8_prompt_attention(q, k, v, tq, tk, o=o)
    for i in (0, 2):
        R.assert_within(o[cq[i]:cq[i + 1]], ref[0][cq[i]:cq[i + 1]], ref[1][cq[i]:cq[i + 1]], f"sequence {i}")
    assert (o[cq[-1]:] == 3.0).all()


@pytest.mark.parametrize("cq,ck", [([0, 50, 40, 100], [0, 50, 60, 100]), ([0, 50, 60, 140], [0, 50, 60, 100]),
                                   ([0, 50, 60, 100], [0, 50, 60, 140]), ([-5, 50, 60, 100], [0, 50, 60, 100]),
                                   ([0, 50, 60, 100], [0, 50, 40, 100])])
def test_malformed_sequences_are_skipped_and_reported(q8, cq, ck):
    H, Hkv, d = 4, 2, 64
    q, k, v = _rand(1, 100, H, d), _rand(2, 100, Hkv, d), _rand(3, 100, Hkv, d)
    t = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    o = torch.full_like(q, 3.0)
    q8.q8_prompt_attention(q, k, v, t(cq), t(ck), o=o)
    assert q8.q8_device_error() == 512
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("at", [0, 511, 512, 2999])
def test_a_malformed_sequence_among_many_is_reported(q8, at):
    B, d = 3000, 64
    q = _rand(1, B, 1, d)
    t = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ck = t.clone()
    o = q8.q8_prompt_attention(q, q, q, t, ck)
    assert q8.q8_device_error() == 0
    assert torch.equal(o, q)  # one key each: its value
    ck[at] = ck[at + 1] + 1
    q8.q8_prompt_attention(q, q, q, t, ck)
    assert q8.q8_device_error() == 512


def test_two_calls_and_two_graphs_at_once(q8):
    """The same shapes on two streams together, then two captured graphs replayed together:
    each call has its own workspace."""
    H, Hkv, d = 8, 2, 128
    sets = []
    for s in range(2):
        (cq, tq), (ck, tk) = _cum([1, 3]), _cum([20000, 900])
        sets.append((_rand(s, 4, H, d), _rand(s + 10, ck[-1], Hkv, d), _rand(s + 20, ck[-1], Hkv, d), tq, tk))
    want = [q8.q8_prompt_attention(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for a, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(q8.q8_prompt_attention(*a))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs, outs = [], []
    for a, st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(q8.q8_prompt_attention(*a))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(NAN)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    # other lengths in the same graph: they live on the device
    sets[0][4].copy_(torch.tensor([0, 700, 1200], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    a = sets[0]
    R.assert_within(outs[0], *R.prompt(a[0], a[1], a[2], [0, 1, 4], [0, 700, 1200]), "replayed with other lengths")


def test_same_result_every_time(q8):
    (cq, tq), (ck, tk) = _cum([400, 1, 30]), _cum([400, 5000, 31])
    a = _rand(1, cq[-1], 16, 128), _rand(2, ck[-1], 4, 128), _rand(3, ck[-1], 4, 128), tq, tk
    first = q8.q8_prompt_attention(*a)
    for _ in range(5):
        assert torch.equal(q8.q8_prompt_attention(*a), first)


def test_keys_behind_4_gigabytes(q8):
    """Keys 2^25 elements apart: offsets beyond 32 bits."""
    n, d = 130, 64
    try:
        big = torch.empty((n - 1) * (1 << 25) + 256, dtype=BF16, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    k, v = big.as_strided((n, 1, d), (1 << 25, d, 1)), big.as_strided((n, 1, d), (1 << 25, d, 1), 128)
    k.copy_(_rand(1, n, 1, d))
    v.copy_(_rand(2, n, 1, d))
    q = _rand(3, n, 2, d)
    c, t = _cum([n])
    o = q8.q8_prompt_attention(q, k, v, t)
    assert torch.equal(o, q8.q8_prompt_attention(q, k.contiguous(), v.contiguous(), t))
    R.assert_within(o, *R.prompt(q, k, v, c, c))
    own = big.as_strided((2, 65, 1, d), (65 << 25, 1 << 25, d, 1)), big.as_strided((2, 65, 1, d), (65 << 25, 1 << 25, d, 1), 128)
    ln = torch.tensor([65, 33], dtype=torch.int32, device="cuda")
    o = q8.q8_prefix_attention(q[:2], k, v, *own, ln)
    R.assert_within(o, *R.prefix(q[:2], k, v, *own, [65, 33]))


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (4, 1, 128), (16, 16, 64)])
@pytest.mark.parametrize("B,longest", [(33, 9), (1025, 3), (1500, 70)])
def test_many_sequences(q8, B, longest, H, Hkv, d):
    """More sequences than one round of the search tells apart, empty ones among them, and far
    more work items than the GPU has SMs."""
    _prompt(q8, [(i * 7) % (longest + 1) for i in range(B)], [(i * 7) % (longest + 1) for i in range(B)], H, Hkv, d,
            seed=B)


def test_few_new_tokens_among_many_empty_sequences(q8):
    """Split keys with more items than SMs: most of them belong to sequences without a query."""
    nq, nk = [0] * 700, [0] * 700
    nq[3], nk[3], nq[350], nk[350], nq[699], nk[699] = 1, 9000, 5, 4000, 2, 20000
    nk[5] = 77
    _prompt(q8, nq, nk, 8, 2, 128, seed=8)
    _prompt(q8, nq, nk, 4, 4, 64, seed=8)


def test_every_shape_again_and_again(q8):
    """Calls of different cuts behind one another on one stream, each as it is alone."""
    calls = []
    for s, (nq, nk, H, Hkv, d) in enumerate([([900, 70], [900, 70], 32, 8, 128), ([1], [9000], 8, 2, 128),
                                             ([40] * 30, [40] * 30, 16, 16, 64), ([3, 2], [4000, 10], 8, 1, 64)]):
        q, k, v, tq, tk, o = _prompt(q8, nq, nk, H, Hkv, d, seed=s)
        calls.append((q8.q8_prompt_attention, (q, k, v, tq, tk), o))
    for B, P, cap in ((1, 300, 60), (20, 3000, 100), (5, 9000, 3000), (70, 0, 40)):
        a = _prefix(q8, B, P, cap, [(i * 29 + cap) % (cap + 1) for i in range(B)], 8, 2, 128, seed=B)
        calls.append((q8.q8_prefix_attention, a[:6], a[6]))
    for i in range(40):
        got = [f(*a) for f, a, _ in calls]
        for j, (x, (_, _, want)) in enumerate(zip(got, calls)):
            assert torch.equal(x, want), (i, j)
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("n", [300, 5000])
def test_scores_of_minus_infinity_weigh_nothing(q8, n):
    """Visible keys whose score is below binary32: the others carry the softmax."""
    H, Hkv, d = 4, 2, 128
    q, k, v = _rand(1, 3, H, d), _rand(2, n, Hkv, d), _rand(3, n, Hkv, d)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[:160], bad[200:203] = True, True
    q[..., 0], k[..., 0] = 2.0 ** 100, 0.0
    good_k, good_v = k[~bad], v[~bad]
    k[bad, :, 0] = -2.0 ** 100
    ln = torch.tensor([n] * 3, dtype=torch.int32, device="cuda")
    z = k[:0]
    m = good_k.shape[0]
    q0, one = q.clone(), lambda x: x[None].expand(3, *x.shape)
    q0[..., 0] = 0  # the same scores over the good keys: their first channel is 0
    want = R.prefix(q0, z, z, one(good_k), one(good_v), [m] * 3)
    R.assert_within(q8.q8_prefix_attention(q, z, z, one(k), one(v), ln), *want, "own keys")
    R.assert_within(q8.q8_prefix_attention(q, k, v, one(z), one(z), ln * 0), *want, "shared keys")
    for i in range(3):
        got = q8.q8_prompt_attention(q[i:i + 1], k, v, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                     torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        R.assert_within(got, want[0][i:i + 1], want[1][i:i + 1], "prompt")


def test_work_on_a_stream_that_is_not_current(q8):
    """New outputs and workspaces belong to the stream of the call: what the current stream does
    with freed memory does not reach them, nor they it."""
    (cq, tq), (ck, tk) = _cum([1]), _cum([50000])
    a = _rand(1, 1, 8, 128), _rand(2, 50000, 2, 128), _rand(3, 50000, 2, 128), tq, tk
    want = q8.q8_prompt_attention(*a)
    need = q8.q8_prompt_attention_workspace_size(1, 1, 50000, 8, 2, 128)
    assert need > 0
    side = torch.cuda.Stream()
    x = torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(10_000_000)  # the current stream still writes x when the side stream is done
    x.fill_(NAN)
    del x
    got = q8.q8_prompt_attention(*a, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    o = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)  # the workspace is written when the call is long over
    q8.q8_prompt_attention(*a, o=o, stream=side)
    y = torch.zeros(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(o, want) and (y == 0).all()


def test_empty_prompts(q8):
    z = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    t = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    assert q8.q8_prompt_attention(z, z, z, t([0])).shape == z.shape
    assert q8.q8_prompt_attention(z, z, z, t([0, 0, 0])).shape == z.shape
    q = _rand(1, 5, 4, 64)
    assert (q8.q8_prompt_attention(q, z, z, t([0, 5]), t([0, 0])) == 0).all()
    o = torch.full_like(q, 2.0)
    q8.q8_prompt_attention(q, q, q, t([0]), o=o)  # no sequence: nothing is written
    assert (o == 2.0).all()
    assert q8.q8_device_error() == 0


# ---- shared prefix -------------------------------------------------------------------------
def _prefix(q8, B, P, cap, lens, H, Hkv, d, seed=0, gain=1.0, **kw):
    q = _rand(seed, B, H, d, gain=gain)
    kp, vp = _rand(seed + 1, P, Hkv, d), _rand(seed + 2, P, Hkv, d)
    ko, vo = _rand(seed + 3, B, cap, Hkv, d), _rand(seed + 4, B, cap, Hkv, d)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):  # rows behind a request's length are not read
        ko[b, n:], vo[b, n:] = NAN, NAN
    o = q8.q8_prefix_attention(q, kp, vp, ko, vo, ln, **kw)
    R.assert_within(o, *R.prefix(q, kp, vp, ko, vo, lens, kw.get("scale")), f"B={B} P={P} {lens[:9]} {H}/{Hkv} d={d}")
    assert q8.q8_device_error() == 0
    return q, kp, vp, ko, vo, ln, o


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("B,P,cap,lens", [
    (1, 1, 1, [1]), (1, 0, 5, [3]), (1, 700, 9, [0]), (3, 0, 1, [0, 1, 0]), (2, 129, 130, [128, 129]),
    (5, 64, 64, [64, 63, 1, 0, 33]), (37, 300, 70, [(7 * i) % 71 for i in range(37)]), (2, 5000, 0, [0, 0]),
    (4, 127, 700, [700, 513, 512, 511])])
def test_prefix_batches(q8, B, P, cap, lens, H, Hkv, d):
    _prefix(q8, B, P, cap, lens, H, Hkv, d, seed=B + P)


@pytest.mark.parametrize("G,Hkv,d", [(128, 1, 64), (100, 1, 128), (65, 2, 128), (16, 2, 128), (17, 1, 64)])
def test_prefix_with_wide_groups(q8, G, Hkv, d):
    _prefix(q8, 3, 200, 90, [90, 0, 17], G * Hkv, Hkv, d, seed=G)


def test_no_key_at_all_gives_zero(q8):
    *_, o = _prefix(q8, 3, 0, 4, [0, 2, 0], 4, 2, 64)
    assert (o[0] == 0).all() and (o[2] == 0).all() and (o[1] != 0).any()
    *_, o = _prefix(q8, 3, 0, 0, [0, 0, 0], 4, 2, 128)
    assert (o == 0).all()


def test_long_prefix_and_large_batches(q8):
    _prefix(q8, 2, 70001, 300, [300, 1], 8, 2, 128)
    _prefix(q8, 300, 1000, 40, [i % 41 for i in range(300)], 4, 1, 128)
    _prefix(q8, 1, 60, 30011, [30011], 8, 2, 128)


@pytest.mark.parametrize("B,P,cap", [(1, 640, 640), (1, 641, 640), (1, 1024, 1024), (4, 1024, 200), (4, 1025, 200), (70, 58, 900), (64, 64, 320), (64, 64, 321),
                                     (70, 0, 1030), (300, 0, 70), (2, 1, 2047), (2, 1, 2048)])
@pytest.mark.parametrize("H,Hkv,d", [(8, 8, 64), (20, 1, 128)])
def test_both_sides_of_the_single_launch(q8, B, P, cap, H, Hkv, d):
    _prefix(q8, B, P, cap, [(i * 131 + cap) % (cap + 1) for i in range(B)], H, Hkv, d, seed=B)


@pytest.mark.parametrize("gain", [0.0, 8.0, 40.0])
def test_prefix_flat_and_sharp_scores(q8, gain):
    _prefix(q8, 40, 900, 300, [(i * 37) % 301 for i in range(40)], 8, 2, 128, gain=gain)
    _prefix(q8, 2, 900, 300, [300, 77], 8, 2, 128, gain=gain, scale=0.2)


def test_prefix_layouts(q8):
    B, P, cap, H, Hkv, d = 9, 333, 50, 6, 2, 128
    lens = [0, 50, 1, 2, 3, 49, 20, 33, 7]
    q, kp, vp, ko, vo, ln, o = _prefix(q8, B, P, cap, lens, H, Hkv, d)
    m3, m4 = (lambda y: y.transpose(0, 1).contiguous().transpose(0, 1)), (lambda y: y.transpose(1, 2).contiguous().transpose(1, 2))
    om = m3(torch.full_like(q, NAN))
    q8.q8_prefix_attention(m3(q), m3(kp), m3(vp), m4(ko), m4(vo), ln, o=om)
    assert torch.equal(om, o)
    both = torch.stack((kp, vp), 1)  # keys and values of a token side by side
    mine = torch.stack((ko, vo), 2)
    assert torch.equal(q8.q8_prefix_attention(q, both[:, 0], both[:, 1], mine[:, :, 0], mine[:, :, 1], ln), o)
    kq, vq = ko[:1].expand_as(ko), vo[:1].expand_as(vo)  # one own cache for all, stride 0
    n1 = torch.full((B,), 0, dtype=torch.int32, device="cuda")
    assert torch.equal(q8.q8_prefix_attention(q, kp, vp, kq, vq, n1), q8.q8_prefix_attention(q, kp, vp, ko, vo, n1))


def test_lengths_outside_the_cache_are_clamped_and_reported(q8):
    B, P, cap, H, Hkv, d = 3, 100, 20, 4, 2, 128
    q, kp, vp = _rand(1, B, H, d), _rand(2, P, Hkv, d), _rand(3, P, Hkv, d)
    ko, vo = _rand(4, B, cap, Hkv, d), _rand(5, B, cap, Hkv, d)
    ln = torch.tensor([-3, 5, 21], dtype=torch.int32, device="cuda")
    o = q8.q8_prefix_attention(q, kp, vp, ko, vo, ln)
    assert q8.q8_device_error() == 512
    R.assert_within(o, *R.prefix(q, kp, vp, ko, vo, [0, 5, 20]))
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("where", ["q", "ko", "vo"])
def test_a_request_does_not_reach_its_neighbours(q8, where):
    B, P, cap, H, Hkv, d = 40, 150, 33, 4, 2, 128
    lens = [(i * 5) % 34 for i in range(B)]
    q, kp, vp, ko, vo, ln, o = _prefix(q8, B, P, cap, lens, H, Hkv, d)
    q2, ko2, vo2 = q.clone(), ko.clone(), vo.clone()
    {"q": q2, "ko": ko2, "vo": vo2}[where][5] = NAN
    o2 = q8.q8_prefix_attention(q2, kp, vp, ko2, vo2, ln)
    keep = torch.arange(B, device="cuda") != 5
    assert torch.equal(o2[keep], o[keep])


def test_prefix_streams_and_graphs(q8):
    args = [_prefix(q8, 12, 3000, 200, [(i * 19 + s) % 201 for i in range(12)], 8, 2, 128, seed=s) for s in (0, 100)]
    streams = [torch.cuda.Stream() for _ in args]
    graphs, outs = [], []
    for a, st in zip(args, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(q8.q8_prefix_attention(*a[:6]))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(NAN)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, a[6]) for o, a in zip(outs, args))
    a = args[0]
    a[5].copy_(torch.tensor([0] * 6 + [200] * 6, dtype=torch.int32))  # the next step's lengths
    ko, vo = (torch.nan_to_num(x, 0.5) for x in a[3:5])
    a[3].copy_(ko)
    a[4].copy_(vo)
    graphs[0].replay()
    torch.cuda.synchronize()
    R.assert_within(outs[0], *R.prefix(*a[:5], [0] * 6 + [200] * 6), "replayed with other lengths")


# ---- the entry points together -------------------------------------------------------------
def test_own_workspace(q8):
    (cq, tq), (ck, tk) = _cum([1]), _cum([50000])
    a = _rand(1, 1, 8, 128), _rand(2, 50000, 2, 128), _rand(3, 50000, 2, 128), tq, tk
    need = q8.q8_prompt_attention_workspace_size(1, 1, 50000, 8, 2, 128)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    o = q8.q8_prompt_attention(*a, workspace=ws[:need])
    assert torch.equal(o, q8.q8_prompt_attention(*a)) and (ws[need:] == 0xAB).all()
    B, P, cap = 3, 20000, 100
    b = (_rand(1, B, 8, 128), _rand(2, P, 2, 128), _rand(3, P, 2, 128), _rand(4, B, cap, 2, 128),
         _rand(5, B, cap, 2, 128), torch.tensor([3, 0, 100], dtype=torch.int32, device="cuda"))
    need = q8.q8_prefix_attention_workspace_size(B, P, cap, 8, 2, 128)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    o = q8.q8_prefix_attention(*b, workspace=ws[:need])
    assert torch.equal(o, q8.q8_prefix_attention(*b)) and (ws[need:] == 0xAB).all()
    if need:
        with pytest.raises(q8.Q8Error, match="Q8_ERR_NOMEM"):
            q8.q8_prefix_attention(*b, workspace=ws[:need - 16])


def test_refusals(q8):
    q, k = _rand(1, 10, 4, 128), _rand(2, 10, 2, 128)
    t = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="k"):
        q8.q8_prompt_attention(q, k.float(), k, t)
    with pytest.raises(TypeError, match="cu_q"):
        q8.q8_prompt_attention(q, k, k, t.long())
    with pytest.raises(ValueError, match="cu_k"):
        q8.q8_prompt_attention(q, k, k, t, t[:1])
    with pytest.raises(ValueError, match="v"):
        q8.q8_prompt_attention(q, k, k[:9], t)
    with pytest.raises(ValueError, match="channels"):
        q8.q8_prompt_attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, t)
    for bad in (torch.empty(10, 4, 96, dtype=BF16, device="cuda"),):
        with pytest.raises(q8.Q8Error, match="Q8_ERR_SHAPE"):
            q8.q8_prompt_attention(bad, bad[:, :2], bad[:, :2], t)
    with pytest.raises(q8.Q8Error, match="Q8_ERR_SHAPE"):
        q8.q8_prompt_attention(q[:, :3], k, k, t)
    with pytest.raises(q8.Q8Error, match="Q8_ERR_VALUE"):
        q8.q8_prompt_attention(q, k, k, t, scale=-1.0)
    odd = torch.empty(10, 4 * 128 + 4, dtype=BF16, device="cuda")[:, 4:].view(10, 4, 128)
    with pytest.raises(q8.Q8Error, match="Q8_ERR_ALIGN"):
        q8.q8_prompt_attention(odd, k, k, t)
    with pytest.raises(q8.Q8Error, match="Q8_ERR_SHAPE"):
        q8.q8_prompt_attention(q, k, k, t, o=torch.empty(1, 4, 128, dtype=BF16, device="cuda").expand(10, 4, 128))
    ko = _rand(3, 10, 5, 2, 128)
    with pytest.raises(ValueError, match="k_own"):
        q8.q8_prefix_attention(q, k, k, ko[:9], ko, t[:1].expand(10))
    with pytest.raises(ValueError, match="own_len"):
        q8.q8_prefix_attention(q, k, k, ko, ko, t)


def test_a_layer_from_prompt_to_next_tokens(q8):
    """Projection -> heads' norm and rotation -> packed prompts; then one more token of two
    requests behind the shared first prompt, its keys appended to the requests' own caches."""
    H, Hkv, d, K = 8, 2, 64, 256
    n = [150, 40, 25]  # a shared instruction, and what two requests add to it
    T = sum(n)
    g = torch.Generator(device="cuda").manual_seed(11)
    W = torch.randn((H + 2 * Hkv) * d, K, generator=g, device="cuda") * 0.05
    Wq, Wd = q8.q8_quantize_weights(W)
    inv = 1e4 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    qw, kw = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))

    def project(x, pos):
        y = q8.q8_linear_fused(x, Wq, Wd, out_dtype=BF16)
        q, k, v = (y[:, a * d:b * d].view(-1, b - a, d) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
        q, k = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
        return q, k, v

    x = torch.randn(T + 2, K, generator=g, device="cuda").to(BF16)
    pos = torch.cat((torch.arange(150), torch.arange(150, 190), torch.arange(150, 175))).to("cuda", torch.int32)
    q, k, v = project(x[:T].contiguous(), pos)
    # the requests' own tokens see the instruction too: their keys are packed behind a copy of it
    ks = torch.cat((k[:150], k[:150], k[150:190], k[:150], k[190:]))
    vs = torch.cat((v[:150], v[:150], v[150:190], v[:150], v[190:]))
    (cq, tq), (ck, tk) = _cum(n), _cum([150, 190, 175])
    o = q8.q8_prompt_attention(q, ks, vs, tq, tk)
    R.assert_within(o, *R.prompt(q, ks, vs, cq, ck), "prompts")
    # the next token of each request
    q1, k1, v1 = project(x[T:].contiguous(), torch.tensor([190, 175], dtype=torch.int32, device="cuda"))
    ko, vo = (torch.full((2, 64, Hkv, d), NAN, dtype=BF16, device="cuda") for _ in range(2))
    for c, new, y in ((ko, k1, k), (vo, v1, v)):
        c[0, :40], c[1, :25] = y[150:190], y[190:]
        c[torch.arange(2), torch.tensor([40, 25])] = new
    ln = torch.tensor([41, 26], dtype=torch.int32, device="cuda")
    got = q8.q8_prefix_attention(q1, k[:150], v[:150], ko, vo, ln)
    R.assert_within(got, *R.prefix(q1, k[:150], v[:150], ko, vo, [41, 26]), "next tokens")
    # the same tokens as single-query prompts
    ks = torch.cat((k[:150], ko[0, :41], k[:150], ko[1, :26]))
    vs = torch.cat((v[:150], vo[0, :41], v[:150], vo[1, :26]))
    (_, tq), (ck, tk) = _cum([1, 1]), _cum([191, 176])
    R.assert_within(q8.q8_prompt_attention(q1, ks, vs, tq, tk), *R.prompt(q1, ks, vs, [0, 1, 2], ck), "as prompts")
    assert q8.q8_device_error() == 0


def test_a_decode_step_captured_once(q8):
    """Rotation in place, the new key into the cache, attention behind the prefix: one graph,
    replayed for the next tokens with positions and lengths advanced on the device."""
    B, P, cap, H, Hkv, d = 5, 300, 40, 8, 2, 128
    kp, vp = _rand(1, P, Hkv, d), _rand(2, P, Hkv, d)
    ko, vo = (torch.full((B, cap, Hkv, d), NAN, dtype=BF16, device="cuda") for _ in range(2))
    inv = 1e6 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    x = torch.empty(B, H + 2 * Hkv, d, dtype=BF16, device="cuda")  # the projection's rows
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    ln = torch.tensor([0, 3, 1, 0, 7], dtype=torch.int32, device="cuda")
    for c, s in ((ko, 3), (vo, 4)):
        for b, n in enumerate(ln.tolist()):
            c[b, :n] = _rand(s + 10 * b, n, Hkv, d)
    rows = torch.arange(B, device="cuda")

    def step():
        q8.q8_qk_norm_rope(q, k, ln + P, inv, q_out=q, k_out=k)
        at = ln.long()
        ko[rows, at] = k
        vo[rows, at] = v
        ln.add_(1)
        return q8.q8_prefix_attention(q, kp, vp, ko, vo, ln)

    saved = [t.clone() for t in (ko, vo, ln)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(_rand(50, *x.shape))
        step()
    torch.cuda.synchronize()
    for t, s in zip((ko, vo, ln), saved):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = step()
    for i in range(6):
        new = _rand(60 + i, *x.shape)
        x.copy_(new)
        before = ln.tolist()
        g.replay()
        torch.cuda.synchronize()
        assert ln.tolist() == [n + 1 for n in before]
        pos = torch.tensor(before, device="cuda", dtype=torch.int32) + P
        R.assert_within(q, *R.norm_rope(new[:, :H], pos, inv, None, 1e-6, False), "rotated")
        R.assert_within(o, *R.prefix(q, kp, vp, ko, vo, ln.tolist()), f"step {i}")
    assert q8.q8_device_error() == 0
