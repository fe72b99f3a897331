"""The paged 4-bit cache without a GPU: refusals of the C ABI and of the binding, which come before
anything is launched, and the tests' own plain forms."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
from tests import kv4_ref as K  # noqa: E402

P = ctypes.c_void_p
FAKE = 0x10000  # aligned, non-null, never dereferenced: every call below fails validation first
I64 = ctypes.c_int64
NULL, SHAPE, ALIGN, DTYPE, VALUE = 1, 2, 3, 4, 9
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


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


def _strides(*v):
    return (I64 * len(v))(*v)


def test_table_rejects_bad_arguments(L):
    # 0 positions 1 axes 2 inv_freq 3 axis 4 table 5 T 6 half 7 stream
    call = _caller(L.q8_rope_table, [P(FAKE), 3, P(FAKE), P(FAKE), P(FAKE), 5, 32, None])
    for bad in (dict(_5=-1), dict(_1=0), dict(_6=-8), dict(_6=12), dict(_6=1032), dict(_5=1 << 31), dict(_1=1 << 31)):
        assert call(**bad) == SHAPE, bad
    for i in (0, 2, 4):
        assert call(**{f"_{i}": None}) == NULL, i
    for i, off in ((0, 2), (2, 4), (3, 1), (4, 8)):
        assert call(**{f"_{i}": P(FAKE + off)}) == ALIGN, i


# the cache's arguments: page stride, pages, page
CACHE = (2 * 2 * 36 * 128, 5, 64)
BAD_CACHE = [(dict(pages=-1), SHAPE), (dict(page=0), SHAPE), (dict(page=48), SHAPE), (dict(page=1 << 17), SHAPE),
             (dict(stride=CACHE[0] - 16), SHAPE), (dict(stride=-16), SHAPE), (dict(stride=CACHE[0] + 8), ALIGN),
             (dict(pages=1 << 26), SHAPE), (dict(stride=1 << 40), SHAPE)]


def _cache_args(at, bad):
    return {f"_{at + i}": bad[k] for i, k in enumerate(("stride", "pages", "page")) if k in bad}


def test_append_rejects_bad_arguments(L):
    # 0 q 1 k 2 v 3 type 4 strides 5 qw 6 kw 7 eps 8 table 9 rot 10 interleaved 11 slots 12 cache 13-15 stride, pages, page
    # 16 q_out 17 T 18 H 19 Hkv 20 d 21 stream
    call = _caller(L.q8_kv4_append, [P(FAKE), P(FAKE), P(FAKE), 1, None, P(FAKE), P(FAKE), 1e-6, P(FAKE), 64, 0, P(FAKE),
                                     P(FAKE), *CACHE, P(FAKE), 4, 4, 2, 128, None])
    assert call(_3=2) == DTYPE
    for bad in (dict(_17=-1), dict(_18=-1), dict(_19=-1), dict(_20=96), dict(_9=-16), dict(_9=8), dict(_9=144),
                dict(_17=1 << 31), dict(_17=1 << 30), dict(_19=1 << 17)):
        assert call(**bad) == SHAPE, bad
    for bad, want in BAD_CACHE:
        assert call(**_cache_args(13, bad)) == want, bad
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert call(_7=eps) == VALUE
    for i in (0, 1, 2, 8, 11, 12, 16):
        assert call(**{f"_{i}": None}) == NULL, i
    for i in (0, 1, 2, 5, 6, 8, 12, 16):
        assert call(**{f"_{i}": P(FAKE + 8)}) == ALIGN, i
    assert call(_11=P(FAKE + 2)) == ALIGN
    for st, want in (((508, 256, 256, 512), ALIGN), ((512, -8, 256, 512), SHAPE), ((512, 256, 1 << 38, 512), SHAPE),
                     ((512, 256, 256, 504), SHAPE), ((512, 256, 256, 0), SHAPE), ((512, 260, 256, 512), ALIGN)):
        assert call(_4=_strides(*st)) == want, st
    if not torch.cuda.is_available():  # repeated inputs, no queries, no rotation, no norm: these pass
        assert call(_4=_strides(0, 0, 0, 512)) in (6, 7)
        assert call(_0=None, _16=None, _18=0, _5=None, _6=None, _7=0.0, _8=None, _9=0) in (6, 7)


def test_gather_rejects_bad_arguments(L):
    # 0 cache 1-3 stride, pages, page 4 table 5 width 6 first 7 cu 8 k 9 v 10 type 11 B 12 T 13 Hkv 14 d 15 stream
    call = _caller(L.q8_kv4_gather, [P(FAKE), *CACHE, P(FAKE), 3, P(FAKE), P(FAKE), P(FAKE), P(FAKE), 1, 2, 10, 2, 128, None])
    assert call(_10=2) == DTYPE
    for bad in (dict(_11=-1), dict(_12=-1), dict(_13=-1), dict(_14=80), dict(_5=-1), dict(_5=1 << 26), dict(_12=1 << 31),
                dict(_12=1 << 30, _13=2)):
        assert call(**bad) == SHAPE, bad
    for bad, want in BAD_CACHE:
        assert call(**_cache_args(1, bad)) == want, bad
    for i in (0, 4, 7, 8, 9):
        assert call(**{f"_{i}": None}) == NULL, i
    for i, off in ((0, 8), (4, 2), (6, 1), (7, 2), (8, 4), (9, 8)):
        assert call(**{f"_{i}": P(FAKE + off)}) == ALIGN, i


def test_attention_rejects_bad_arguments(L):
    # 0 q 1 cache 2-4 stride, pages, page 5 table 6 width 7 kv_len 8 cu_q 9 o 10 B 11 Tq 12 H 13 Hkv 14 d 15 scale
    # 16 strides 17 workspace 18 bytes 19 stream
    call = _caller(L.q8_kv4_attention, [P(FAKE), P(FAKE), *CACHE, P(FAKE), 3, P(FAKE), P(FAKE), P(FAKE), 2, 6, 4, 2, 128, 0.1,
                                        None, None, 0, None])
    for bad in (dict(_10=-1), dict(_11=-1), dict(_12=3), dict(_13=0), dict(_14=80), dict(_12=258), dict(_6=-1), dict(_6=1 << 26),
                dict(_11=1 << 31), dict(_11=1 << 30), dict(_8=None), dict(_11=1 << 28, _6=1 << 18)):
        assert call(**bad) == SHAPE, bad
    for bad, want in BAD_CACHE:
        assert call(**_cache_args(2, bad)) == want, bad
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(_15=s) == VALUE
    for i in (0, 1, 5, 7, 9):
        assert call(**{f"_{i}": None}) == NULL, i
    for i, off in ((0, 8), (1, 8), (5, 2), (7, 1), (8, 2), (9, 8), (17, 8)):
        assert call(**{f"_{i}": P(FAKE + off)}) == ALIGN, i
    ok = [512, 128, 512, 128]
    for i, v, want in ((0, -8, SHAPE), (0, 0, SHAPE), (1, 0, SHAPE), (1, 132, ALIGN), (2, 504, SHAPE), (3, 64, SHAPE),
                       (0, 1 << 38, SHAPE)):
        st = list(ok)
        st[i] = v
        assert call(_16=_strides(*st)) == want, (i, v)


def test_empty_calls_need_no_pointers(L):
    assert L.q8_rope_table(None, 1, None, None, None, 0, 32, None) in (0, 6, 7)
    assert L.q8_kv4_append(None, None, None, 1, None, None, None, 0.0, None, 0, 0, None, None, *CACHE, None, 0, 4, 2, 128, None) in (0, 6, 7)
    assert L.q8_kv4_gather(None, *CACHE, None, 3, None, None, None, None, 0, 0, 0, 2, 128, None) in (0, 6, 7)
    assert L.q8_kv4_attention(None, None, *CACHE, None, 3, None, None, None, 0, 0, 4, 2, 128, 0.1, None, None, 0, None) in (0, 6, 7)


def test_sizes(q8):
    assert q8.q8_kv4_attention_workspace_size(2, 3, 64, 4, 3, 128) == 0
    assert q8.q8_kv4_attention_workspace_size(2, 3, 48, 4, 2, 128) == 0
    assert q8.q8_kv4_cache_shape(7, 64, 3, 128) == (7, 3, 2, 36 * 128)
    for page, d in ((48, 128), (0, 128), (64, 96)):
        with pytest.raises(ValueError, match="page"):
            q8.q8_kv4_cache_shape(7, page, 3, d)


def test_binding_refuses_host_tensors_and_wrong_types(q8, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t)  # noqa: E731
    cache, bt, n = z(2, 1, 1, 36 * 64, t=U8), z(4, 2, t=I32), z(4, t=I32)
    kv = z(4, 1, 64)
    with pytest.raises(ValueError, match="positions: must be"):
        q8.q8_rope_table(n, z(32, t=torch.float64))
    with pytest.raises(TypeError, match="positions"):
        q8.q8_rope_table(z(4, t=torch.int64), z(32, t=torch.float64))
    with pytest.raises(TypeError, match="k: expected"):
        q8.q8_kv4_append(z(4, 1, 64, t=torch.float16), kv, cache, n)
    with pytest.raises(ValueError, match="k: must be a CUDA tensor"):
        q8.q8_kv4_append(kv, kv, cache, n)
    with pytest.raises(TypeError, match="q: expected"):
        q8.q8_kv4_attention(z(4, 2, 64, t=F32), cache, bt, n)
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        q8.q8_kv4_attention(z(4, 2, 64), cache, bt, n)
    with pytest.raises(TypeError, match="out_dtype"):
        q8.q8_kv4_gather(cache, bt, z(5, t=I32), 4, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="cache"):
        q8.q8_kv4_gather(cache.view(torch.int8), bt, z(5, t=I32), 4)
    with pytest.raises(ValueError, match="cache: expected shape"):
        q8.q8_kv4_gather(cache[0], bt, z(5, t=I32), 4)
    with pytest.raises(ValueError, match="cache: must be a CUDA tensor"):
        q8.q8_kv4_gather(cache, bt, z(5, t=I32), 4)


def test_a_tile_holds_every_code_once():
    for d in (64, 128, 256):
        kb, ks, vb, vs = K.places(d)
        for at, sh, lo in ((kb, ks, 0), (vb, vs, 18 * d)):
            used = sorted((2 * at + sh // 4).flatten().tolist())
            assert used == list(range(2 * lo, 2 * lo + 32 * d))
        g = torch.Generator().manual_seed(d)
        codes = [torch.randint(0, 16, (3, 32, d), generator=g) for _ in range(2)]
        scales = [torch.rand(3, 32, d // 32, generator=g).to(BF16) for _ in range(2)]
        for x, y in zip(K.unpack(K.pack(*codes, *scales)), codes + scales):
            assert torch.equal(x, y.to(x.dtype))


def test_the_plain_forms_agree_with_closed_forms():
    """A quantised block is off by at most half a step; one key: o is its value; equal scores: the mean."""
    x = torch.randn(5, 2, 64)
    codes, top = K.quantised(x)
    assert codes.min() >= 1 and codes.max() <= 15
    back = K.values(codes.view(1, 10, 64), (top / 7).view(1, 10, 2)).view(5, 2, 64)
    assert ((back - x).abs() <= (top / 14).repeat_interleave(32, -1) * 1.001).all()
    q = torch.randn(2, 4, 64).to(BF16)
    k, s = torch.zeros(3, 2, 64), torch.ones(3, 2, 2)
    v = torch.randn(3, 2, 64)
    seen = torch.tensor([[True, False, False], [True, True, True]])
    o, tol = K.attention(q, k, v, s, s, seen, 0.125)
    assert torch.allclose(o[0, 3], v[0, 1].double()) and torch.allclose(o[1, 0], v[:, 0].double().mean(0))
    assert (tol >= K.STEP * o.abs()).all()
    z = K.turned(torch.ones(1, 1, 64), None, torch.stack((torch.zeros(1, 16), torch.ones(1, 16)), 1), True)
    assert torch.equal(z[0, 0, :4], torch.tensor([-1.0, 1.0, -1.0, 1.0])) and torch.equal(z[0, 0, 32:], torch.ones(32))
