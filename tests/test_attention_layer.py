"""The attention layer's entry points without a GPU: refusals of the C ABI and of the binding,
which come before anything is launched, and the tests' own binary64 forms."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402

P = ctypes.c_void_p
FAKE = 0x10000  # aligned, non-null, never dereferenced: every call below fails validation first
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def q8():
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    return m


@pytest.fixture(scope="module")
def L(q8):
    return q8.lib()


def _caller(f, ok):
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


def _strides(n, **kw):
    a = (I64 * n)(*[0] * n)
    for i, v in kw.items():
        a[int(i[1:])] = v
    return a


NULL, SHAPE, ALIGN, DTYPE, VALUE = 1, 2, 3, 4, 9


def test_qk_norm_rope_rejects_bad_arguments(L):
    #     0 q      1 k     2 type 3 qs 4 ks  5 qw    6 kw   7 eps 8 positions 9 inv_freq
    call = _caller(L.q8_qk_norm_rope, [
        P(FAKE), P(FAKE), 1, 512, 512, P(FAKE), P(FAKE), 1e-6, P(FAKE), P(FAKE),
        # 10 rot 11 interleaved 12 q_out 13 k_out 14 qos 15 kos 16 T 17 H 18 Hkv 19 d 20 stream
        64, 0, P(FAKE), P(FAKE), 256, 128, 4, 4, 2, 64, None])
    assert call(_2=2) == DTYPE
    for bad in (dict(_16=-1), dict(_17=-1), dict(_18=-1), dict(_19=8), dict(_19=72), dict(_19=272),
                dict(_10=-16), dict(_10=8), dict(_10=80), dict(_3=-8), dict(_14=248), dict(_15=120),
                dict(_16=1 << 31), dict(_3=1 << 40)):
        assert call(**bad) == SHAPE, bad
    for i in (0, 1, 8, 9, 12, 13):
        assert call(**{f"_{i}": None}) == NULL, i
    for i in (0, 1, 5, 6, 12, 13):
        assert call(**{f"_{i}": P(FAKE + 8)}) == ALIGN, i
    assert call(_8=P(FAKE + 2)) == ALIGN and call(_9=P(FAKE + 4)) == ALIGN
    assert call(_3=516) == ALIGN and call(_4=516) == ALIGN and call(_14=260) == ALIGN and call(_15=132) == ALIGN
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert call(_7=eps) == VALUE
        assert call(_5=None, _7=eps) == VALUE
        if not torch.cuda.is_available():  # these arguments pass: no norm, eps is not read
            assert call(_5=None, _6=None, _7=eps) in (6, 7)


def test_prompt_attention_rejects_bad_arguments(L):
    # 0 q 1 k 2 v 3 cu_q 4 cu_k 5 o 6 B 7 Tq 8 Tk 9 H 10 Hkv 11 d 12 scale 13 strides 14 ws 15 bytes 16 stream
    call = _caller(L.q8_prompt_attention, [P(FAKE)] * 6 + [2, 10, 10, 4, 2, 128, 0.1, None, None, 0, None])
    for bad in (dict(_6=-1), dict(_7=-1), dict(_8=-1), dict(_9=3), dict(_10=0), dict(_11=96), dict(_11=256),
                dict(_9=258, _10=2), dict(_7=1 << 31), dict(_7=1 << 30, _9=8), dict(_6=0x7FFFFFFF)):
        assert call(**bad) == SHAPE, bad
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(_12=s) == VALUE
    for i in range(6):
        assert call(**{f"_{i}": None}) == NULL, i
    for i in (0, 1, 2, 5, 14):
        assert call(**{f"_{i}": P(FAKE + 8)}) == ALIGN, i
    assert call(_3=P(FAKE + 2)) == ALIGN and call(_4=P(FAKE + 1)) == ALIGN
    # strides: negative, too long for the tile copies, not whole 16-byte pieces, rows of o that overlap
    ok = dict(_0=512, _1=128, _2=256, _3=128, _4=256, _5=128, _6=512, _7=128)
    for bad, want in ((dict(_0=-512), SHAPE), (dict(_0=0), SHAPE), (dict(_4=0), SHAPE), (dict(_1=0), SHAPE),
                      (dict(_2=1 << 38), SHAPE), (dict(_3=132), ALIGN), (dict(_0=4), ALIGN),
                      (dict(_6=0), SHAPE), (dict(_6=504), SHAPE), (dict(_7=64), SHAPE), (dict(_6=128, _7=1272), SHAPE)):
        assert call(_13=_strides(8, **{**ok, **bad})) == want, bad
    if not torch.cuda.is_available():  # these arguments pass: o with each head's tokens together
        assert call(_13=_strides(8, **{**ok, "_6": 128, "_7": 1280})) in (6, 7)


def test_prefix_attention_rejects_bad_arguments(L):
    # 0 q 1 kp 2 vp 3 ko 4 vo 5 own_len 6 o 7 B 8 P 9 cap 10 H 11 Hkv 12 d 13 scale 14 strides 15 ws 16 bytes 17 stream
    call = _caller(L.q8_prefix_attention, [P(FAKE)] * 7 + [2, 10, 10, 4, 2, 128, 0.1, None, None, 0, None])
    for bad in (dict(_7=-1), dict(_8=-1), dict(_9=-1), dict(_10=3), dict(_11=0), dict(_12=32), dict(_10=258, _11=2),
                dict(_8=1 << 31), dict(_7=1 << 30, _10=8)):
        assert call(**bad) == SHAPE, bad
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(_13=s) == VALUE
    for i in range(7):
        assert call(**{f"_{i}": None}) == NULL, i
    for i in (0, 1, 2, 3, 4, 6, 15):
        assert call(**{f"_{i}": P(FAKE + 8)}) == ALIGN, i
    assert call(_5=P(FAKE + 2)) == ALIGN
    ok = dict(_0=512, _1=128, _2=256, _3=128, _4=256, _5=128, _6=2560, _7=256, _8=128, _9=2560, _10=256, _11=128,
              _12=512, _13=128)
    for bad, want in ((dict(_6=-8), SHAPE), (dict(_7=257), ALIGN), (dict(_12=504), SHAPE), (dict(_13=0), SHAPE)):
        assert call(_14=_strides(14, **{**ok, **bad})) == want, bad


def test_empty_calls_need_no_pointers(L):
    assert L.q8_prompt_attention(None, None, None, None, None, None, 0, 0, 0, 0, 1, 64, 1.0, None, None, 0, None) in (0, 6, 7)
    assert L.q8_prefix_attention(None, None, None, None, None, None, None, 0, 5, 5, 4, 2, 64, 1.0, None, None, 0,
                                 None) in (0, 6, 7)
    assert L.q8_qk_norm_rope(None, None, 0, 0, 0, None, None, 0.0, None, None, 0, 0, None, None, 0, 0, 0, 4, 2, 64,
                             None) in (0, 6, 7)


def test_workspace_sizes_of_bad_shapes_are_zero(q8):
    assert q8.q8_prompt_attention_workspace_size(1, 10, 10, 4, 3, 128) == 0
    assert q8.q8_prefix_attention_workspace_size(1, -1, 10, 4, 2, 128) == 0


def test_binding_refuses_host_tensors_and_wrong_types(q8, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    cu = z(2, t=torch.int32)
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        q8.q8_prompt_attention(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), cu)
    with pytest.raises(TypeError, match="q: expected torch.bfloat16"):
        q8.q8_prompt_attention(z(4, 2, 64, t=torch.float32), z(4, 1, 64), z(4, 1, 64), cu)
    with pytest.raises(TypeError, match="q"):
        q8.q8_qk_norm_rope(z(4, 2, 64, t=torch.float16), z(4, 1, 64), z(4, t=torch.int32), z(32, t=torch.float64))
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        q8.q8_prefix_attention(z(4, 2, 64), z(9, 1, 64), z(9, 1, 64), z(4, 5, 1, 64), z(4, 5, 1, 64), z(4, t=torch.int32))


def test_the_plain_forms_agree_with_closed_forms():
    """One key: o is its value.  Equal scores: the mean.  A right angle swaps a pair."""
    q, k = torch.randn(3, 2, 4), torch.zeros(3, 1, 4)
    v = torch.randn(3, 1, 4)
    o, tol = R.prompt(q, k, v, [0, 3], [0, 3])
    for i in range(3):
        want = v[:i + 1, 0].double().mean(0)
        assert torch.allclose(o[i, 0], want) and torch.allclose(o[i, 1], want)
    assert (tol >= R.STEP * o.abs()).all()
    p, _ = R.prefix(q[2:], k[:2], v[:2], k[None, 2:], v[None, 2:], [1])
    assert torch.allclose(p[0], o[2])
    o, _ = R.prompt(q, k[:1], v[:1], [0, 3], [0, 1])  # one key, three queries: the last one sees it
    assert (o[:2] == 0).all() and torch.allclose(o[2], v[0].double().expand(2, 4))
    x = torch.randn(1, 1, 16)
    quarter = torch.full((8,), math.pi / 2, dtype=torch.float64)
    y, _ = R.norm_rope(x, torch.tensor([1]), quarter, None, 0.0, False)
    assert torch.allclose(y[0, 0, :8], -x[0, 0, 8:].double()) and torch.allclose(y[0, 0, 8:], x[0, 0, :8].double())
    y, _ = R.norm_rope(x, torch.tensor([5]), quarter, None, 0.0, True)
    assert torch.allclose(y[0, 0, 0::2], -x[0, 0, 1::2].double()) and torch.allclose(y[0, 0, 1::2], x[0, 0, 0::2].double())
    y, _ = R.norm_rope(x, torch.tensor([0]), quarter, torch.full((16,), 2.0), 0.0, False)
    assert abs(float((y ** 2).mean()) - 4.0) < 1e-12
