"""Attention calls at the edge of what the entry points promise: malformed sequences beside good
ones, repeated caches.  Against the binary64 forms of tests/attention_ref.py."""
import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


def _rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _heads(many):
    """(query heads, key heads): few, or a key head for every SM (two query tiles a block)."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return (n, n) if many else (4, 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("cq,ck,bad", [
    ([0, 50, 60, 140], [0, 50, 60, 100], 2), ([0, 50, 60, 100], [0, 50, 60, 140], 2),
    ([-5, 50, 60, 100], [0, 50, 60, 100], 0), ([0, 50, 60, 100], [0, 50, 40, 100], 1),
    ([0, 50, 60, 100], [-7, 50, 60, 100], 0), ([0, 50, 50, 100], [0, 50, 20, 100], 1),
    # few queries, many keys: the keys are split and joined
    ([0, 20, 30, 100], [0, 3000, 2000, 6000], 1), ([0, 20, 30, 100], [0, 3000, 4000, 6001], 2),
    ([0, 20, 30, 101], [0, 3000, 4000, 6000], 2), ([-1, 20, 30, 100], [0, 3000, 4000, 6000], 0)])
def test_a_malformed_sequence_is_skipped_and_its_neighbours_are_not(q8, cq, ck, bad, many, d):
    (H, Hkv), Tq, Tk = _heads(many), 100, 6000 if max(ck) > 200 else 100
    q, k, v = _rand(1, Tq, H, d), _rand(2, Tk, Hkv, d), _rand(3, Tk, Hkv, d)
    o = torch.full_like(q, 3.0)
    q8.q8_prompt_attention(q, k, v, _int(cq), _int(ck), o=o)
    assert q8.q8_device_error() == 512
    hk = sorted({0, Hkv - 1})
    h = [i * (H // Hkv) for i in hk]
    for s in range(3):
        a, b, c, e = cq[s], cq[s + 1], ck[s], ck[s + 1]
        if s == bad:
            assert (o[max(a, 0):b] == 3.0).all()
        else:
            ref, tol = R.prompt(q[a:b, h], k[c:e, hk], v[c:e, hk], [0, b - a], [0, e - c])
            R.assert_within(o[a:b, h], ref, tol, f"sequence {s}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,cap", [(100, 50), (3000, 50), (0, 50), (700, 900)])  # one launch, or three
def test_repeated_caches(q8, P, cap, d):
    """One own cache for all requests, one key head for all heads, of the prefix and of the own
    caches: strides of 0."""
    B, H, Hkv = 9, 6, 2
    lens = [0, cap, 1, 2, 3, cap - 1, 20, 33, 7]
    q, ln = _rand(1, B, H, d), _int(lens)
    kp, vp, ko, vo = _rand(2, P, Hkv, d), _rand(3, P, Hkv, d), _rand(4, B, cap, Hkv, d), _rand(5, B, cap, Hkv, d)
    request = lambda x: x[1:2].expand_as(x)  # noqa: E731
    head = lambda x: x[..., 1:2, :].expand_as(x)  # noqa: E731
    for what, a in (("requests", (kp, vp, request(ko), request(vo))), ("prefix heads", (head(kp), head(vp), ko, vo)),
                    ("own heads", (kp, vp, head(ko), head(vo))),
                    ("all", (head(kp), head(vp), head(request(ko)), head(request(vo)))),
                    ("keys only", (head(kp), vp, request(ko), vo))):
        o = q8.q8_prefix_attention(q, *a, ln)
        R.assert_within(o, *R.prefix(q, *a, lens), what)
        assert torch.equal(o, q8.q8_prefix_attention(q, *(x.contiguous() for x in a), ln)), what
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("many,nq,nk,at", [
    (False, 4, 1, 0), (False, 300, 200, 0), (False, 100, 90, 40), (False, 1600, 1540, 3), (False, 1600, 1540, 1539),
    (True, 4, 1, 0), (True, 300, 200, 0), (True, 200, 60, 59), (True, 255, 127, 0)])
def test_a_query_without_a_key_is_zero_whatever_the_values_are(q8, many, nq, nk, at, value, d):
    """A row of v that is not finite reaches the queries that see it, not the ones that see no
    key (1600 queries, 1540 keys: these are split and joined)."""
    H, Hkv = _heads(many) if nk < 1000 else (1, 1)
    q, k, v = _rand(1, nq, H, d), _rand(2, nk, Hkv, d), _rand(3, nk, Hkv, d)
    v[at] = value
    o = torch.full_like(q, 3.0)
    q8.q8_prompt_attention(q, k, v, _int([0, nq]), _int([0, nk]), o=o)
    assert (o[:nq - nk] == 0).all()
    assert not o[nq - nk + at:].isfinite().any()
    # far enough in front of the row it reaches nothing
    clean = max(nq - nk, nq - nk + at - 255)
    v[at] = 0.0
    want = q8.q8_prompt_attention(q, k, v, _int([0, nq]), _int([0, nk]))
    assert torch.equal(o[:clean], want[:clean])
    assert q8.q8_device_error() == 0
