"""The attention kernels' variants that a call with many heads or many requests takes: two query
tiles a block (prompts whose key heads alone give every SM a block, prefixes with two tiles of
requests for every SM), and the join with one warp a row.  As in tests/test_gpu_attention.py,
against the binary64 forms of tests/attention_ref.py, of some heads or some requests."""
import itertools

import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _rand(seed, *shape, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(BF16)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(n):
    c = [0] + list(itertools.accumulate(n))
    return c, _int(c)


# ---- prompts: as many key heads as SMs, so two tiles a block at any length ---------------------
def _some(Hkv, G):
    """A few key heads and their query heads."""
    hk = sorted({0, Hkv // 2, Hkv - 1})
    return hk, [h * G + g for h in hk for g in range(G)]


def _check(o, q, k, v, cq, ck, G, what, scale=None):
    hk, h = _some(k.shape[1], G)
    R.assert_within(o[:, h], *R.prompt(q[:, h], k[:, hk], v[:, hk], cq, ck, scale), what)


def _inputs(nq, nk, G, d, seed, gain=1.0):
    (cq, tq), (ck, tk) = _cum(nq), _cum(nk)
    Hkv = _sms()
    return (_rand(seed, cq[-1], G * Hkv, d, gain=gain), _rand(seed + 1, ck[-1], Hkv, d),
            _rand(seed + 2, ck[-1], Hkv, d), cq, ck, tq, tk)


def _prompt(q8, nq, nk, G, d, seed=0, gain=1.0):
    q, k, v, cq, ck, tq, tk = _inputs(nq, nk, G, d, seed, gain)
    o = q8.q8_prompt_attention(q, k, v, tq, tk)
    _check(o, q, k, v, cq, ck, G, f"{nq} {nk} G={G} d={d}")
    assert q8.q8_device_error() == 0
    return q, k, v, cq, ck, tq, tk, o


WIDE = [(1, 64), (1, 128), (3, 64), (3, 128)]  # query heads of a key head, channels


@pytest.mark.parametrize("G,d", WIDE)
@pytest.mark.parametrize("n", [[1], [127], [128], [129], [256], [257], [64, 65, 63], [0, 1, 0, 130, 0], [257, 300],
                               [385, 1, 640], [33, 511, 7]])
def test_two_tiles_prompts_of_many_lengths(q8, n, G, d):
    _prompt(q8, n, n, G, d, seed=sum(n))


@pytest.mark.parametrize("G,d", WIDE)
@pytest.mark.parametrize("nq,nk", [([1], [1000]), ([130], [131]), ([3, 200], [900, 201]), ([200, 1], [1041, 128]),
                                   ([129], [700]), ([256, 100], [384, 900])])
def test_two_tiles_behind_a_cache(q8, nq, nk, G, d):
    _prompt(q8, nq, nk, G, d, seed=3)


@pytest.mark.parametrize("G,d", WIDE)
@pytest.mark.parametrize("nq,nk", [([4], [1]), ([300, 5], [200, 0]), ([200], [60]), ([255, 130, 1], [1, 2, 0]),
                                   ([90], [40]), ([3], [0])])
def test_two_tiles_queries_without_a_key(q8, nq, nk, G, d):
    """The first tile of a block, or both, may have no key at all."""
    *_, o = _prompt(q8, nq, nk, G, d, seed=4)
    at = 0
    for a, b in zip(nq, nk):
        assert (o[at:at + max(0, a - b)] == 0).all()
        at += a


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [0.0, 8.0, 40.0])
def test_two_tiles_flat_and_sharp_scores(q8, gain, d):
    _prompt(q8, [260, 31], [500, 31], 1, d, seed=5, gain=gain)


@pytest.mark.parametrize("d", [64, 128])
def test_two_tiles_maximum_rising_along_the_keys(q8, d):
    n = 1100
    q, k, v, cq, ck, tq, _ = _inputs([n], [n], 1, d, 1)
    k = (k.float() * (0.5 + torch.arange(n, device="cuda") / 40)[:, None, None]).to(BF16)
    _check(q8.q8_prompt_attention(q, k, v, tq), q, k, v, cq, ck, 1, "rising")
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_two_tiles_scores_of_minus_infinity(q8, d):
    """Keys whose score is below binary32 weigh nothing, at the beginning and in between."""
    n = 500
    q, k, v, cq, ck, tq, _ = _inputs([1], [n], 1, d, 1)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[:160], bad[200:203] = True, True
    q[..., 0], k[..., 0] = 2.0 ** 100, 0.0
    k[bad, :, 0] = -2.0 ** 100
    q0 = q.clone()
    q0[..., 0] = 0  # the same scores over the good keys: their first channel is 0
    o = q8.q8_prompt_attention(q, k, v, tq, _int([0, n]))
    m = int((~bad).sum())
    _check(o, q0, k[~bad], v[~bad], [0, 1], [0, m], 1, "-inf")


@pytest.mark.parametrize("G,d", WIDE)
@pytest.mark.parametrize("value", [NAN, INF])
def test_two_tiles_a_sequence_does_not_reach_its_neighbours(q8, value, G, d):
    nq, nk = [100, 90, 270], [100, 290, 301]
    q, k, v, cq, ck, tq, tk = _inputs(nq, nk, G, d, 1)
    pad = 40  # rows behind the last sequence
    q, k, v = (torch.cat((x, x[:pad])) for x in (q, k, v))
    clean = [x.clone() for x in (q, k, v)]
    for x, c in ((q, cq), (k, ck), (v, ck)):
        x[c[1]:c[2]] = value
        x[c[-1]:] = value
    o = torch.full_like(q, 3.0)
    q8.q8_prompt_attention(q, k, v, tq, tk, o=o)
    hk, h = _some(_sms(), G)
    ref, tol = R.prompt(clean[0][:, h], clean[1][:, hk], clean[2][:, hk], cq, ck)
    for i in (0, 2):
        R.assert_within(o[cq[i]:cq[i + 1], h], ref[cq[i]:cq[i + 1]], tol[cq[i]:cq[i + 1]], f"sequence {i}")
    assert (o[cq[-1]:] == 3.0).all()
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_two_tiles_layouts(q8, d):
    """Each head's tokens together, rows of a projection, a wider o."""
    n = [100, 1, 311]
    q, k, v, cq, ck, tq, tk, o = _prompt(q8, n, n, 1, d, seed=7)
    major = lambda y: y.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    om = major(torch.full_like(q, NAN))
    q8.q8_prompt_attention(major(q), major(k), major(v), tq, o=om)
    assert torch.equal(om, o)
    rows = torch.cat((q, k, v), 1)
    H = q.shape[1]
    wide = torch.full((cq[-1], H, d + 8), NAN, dtype=BF16, device="cuda")
    q8.q8_prompt_attention(rows[:, :H], rows[:, H:2 * H], rows[:, 2 * H:], tq, o=wide[..., :d])
    assert torch.equal(wide[..., :d], o) and wide[..., d:].isnan().all()


# ---- prefixes of many requests ----------------------------------------------------------------
def _prefix(q8, B, P, cap, H, Hkv, d, seed=0, gain=1.0):
    lens = [(i * 29 + cap) % (cap + 1) for i in range(B)]
    q = _rand(seed, B, H, d, gain=gain)
    kp, vp = _rand(seed + 1, P, Hkv, d), _rand(seed + 2, P, Hkv, d)
    ko, vo = _rand(seed + 3, B, cap, Hkv, d), _rand(seed + 4, B, cap, Hkv, d)
    behind = torch.arange(cap, device="cuda")[None] >= _int(lens)[:, None]
    ko[behind], vo[behind] = NAN, NAN
    o = torch.full((B + 1, H, d), 3.0, dtype=BF16, device="cuda")
    q8.q8_prefix_attention(q, kp, vp, ko, vo, _int(lens), o=o[:B])
    hk, h = _some(Hkv, H // Hkv)
    some = sorted({b for b in (0, 1, 31, 32, 126, 127, 128, 129, 255, 256, 257, B // 2, B - 2, B - 1) if b < B})
    at = torch.tensor(some, device="cuda")
    ref = R.prefix(q[at][:, h], kp[:, hk], vp[:, hk], ko[at][:, :, hk], vo[at][:, :, hk], [lens[b] for b in some])
    R.assert_within(o[at][:, h], *ref, f"B={B} P={P} {H}/{Hkv} d={d}")
    assert (o[B] == 3.0).all() and q8.q8_device_error() == 0
    # requests alone, all heads of them: the same keys in other cuts.  Two results are apart by twice
    # the tolerance of one, in which A is below the largest |v| and the binary32 terms below A / 2^13
    most = max(float(x[~x.isnan()].abs().max()) for x in (vp, vo) if x.numel())
    for b in some[::5]:
        one = q8.q8_prefix_attention(q[b:b + 1], kp, vp, ko[b:b + 1], vo[b:b + 1], _int(lens[b:b + 1])).double()
        assert ((one - o[b].double()).abs() <= 2.1 * R.STEP * (one.abs() + most)).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,P,H,Hkv", [(520, 300, 64, 64), (641, 129, 64, 64), (769, 1000, 64, 64), (330, 257, 128, 32),
                                       (500, 300, 64, 64)])
def test_two_tiles_of_requests(q8, B, P, H, Hkv, d):
    """Two tiles of requests a block (the last case: one tile, below the rule's bound)."""
    _prefix(q8, B, P, 40, H, Hkv, d, seed=B)


@pytest.mark.parametrize("gain", [0.0, 8.0, 40.0])
def test_two_tiles_of_requests_flat_and_sharp_scores(q8, gain):
    _prefix(q8, 520, 700, 9, 64, 64, 64, gain=gain)
    _prefix(q8, 520, 700, 9, 64, 64, 128, gain=gain)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,P,cap,H,Hkv", [(250, 1000, 300, 16, 4), (613, 50, 70, 4, 1), (200, 0, 700, 16, 2)])
def test_join_with_one_warp_a_row(q8, B, P, cap, H, Hkv, d):
    _prefix(q8, B, P, cap, H, Hkv, d, seed=B)
