"""Heads' norm with rotation (q8_qk_norm_rope) against its binary64 form; the tolerance is
derived in tests/attention_ref.py."""
import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


def _freq(rot, theta=1e6):
    return theta ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))


def _inputs(T, H, Hkv, d, dtype, seed=0, far=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, (H + 2 * Hkv) * d, generator=g, device="cuda") *
         torch.exp(torch.randn((H + 2 * Hkv) * d, generator=g, device="cuda"))).to(dtype)
    q, k = x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + far
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    return q, k, pos, w


def _check(out, x, pos, inv, w, eps=1e-6, interleaved=False, what=""):
    R.assert_within(out, *R.norm_rope(x, pos, inv, w, eps, interleaved), what)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,Hkv,d,rot", [
    (1, 32, 8, 128, 128), (1, 1, 1, 16, 16), (3, 5, 5, 64, 64), (7, 6, 2, 80, 32), (33, 12, 4, 256, 64),
    (2, 3, 1, 256, 256), (5, 7, 1, 112, 0), (13, 20, 4, 96, 96), (2, 3, 1, 48, 16), (4, 1, 1, 32, 32), (1, 0, 2, 64, 32),
    (6, 3, 0, 64, 48), (2111, 9, 3, 128, 64)])
def test_matches_the_plain_form(q8, T, H, Hkv, d, rot, dtype, interleaved):
    q, k, pos, (qw, kw) = _inputs(T, H, Hkv, d, dtype, seed=T, far=1000)
    inv = _freq(rot)
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, interleaved=interleaved)
    assert qo.dtype == ko.dtype == BF16 and qo.is_contiguous() and ko.is_contiguous()
    _check(qo, q, pos, inv, qw, interleaved=interleaved, what="q")
    _check(ko, k, pos, inv, kw, interleaved=interleaved, what="k")
    again = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, interleaved=interleaved)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("norms", ["none", "q", "k"])
def test_heads_without_a_norm(q8, norms):
    q, k, pos, (qw, kw) = _inputs(9, 4, 2, 128, BF16)
    inv = _freq(128)
    qw, kw = qw if norms == "q" else None, kw if norms == "k" else None
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, eps=1e-5)
    _check(qo, q, pos, inv, qw, eps=1e-5)
    _check(ko, k, pos, inv, kw, eps=1e-5)


@pytest.mark.parametrize("far", [0, 4095, 262143, 1 << 24, (1 << 31) - 9, -5, -(1 << 31)])
def test_far_positions(q8, far):
    q, k, pos, (qw, kw) = _inputs(8, 2, 1, 128, BF16, far=far)
    inv = _freq(128, 1e4)
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    # the reference's own product is off by 2^-53 of the angle: 2^-22 at the farthest position
    _check(qo, q, pos, inv, qw)
    _check(ko, k, pos, inv, kw)


def test_unusual_frequencies(q8):
    """Zero, subnormal, tiny, negative, above a turn a token: pairs of one head."""
    inv = torch.tensor([0.0, 5e-324, 1e-300, -0.25, 1.0, 3.5, 8.0, 1e-9], device="cuda", dtype=torch.float64)
    q, k, pos, _ = _inputs(40, 1, 1, 16, F32)
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv)
    _check(qo, q, pos, inv, None)
    _check(ko, k, pos, inv, None)


def test_zero_heads_and_large_values(q8):
    q, k, pos, (qw, kw) = _inputs(4, 2, 1, 64, F32)
    q = q.clone()
    q[0] = 0.0
    q[1] *= 1e15
    q[2] *= 1e-12  # the mean square is far below eps
    inv = _freq(64)
    qo, _ = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    assert (qo[0] == 0).all()
    _check(qo, q, pos, inv, qw)


def test_in_place_and_strided_outputs(q8):
    H, Hkv, d, T = 6, 2, 128, 37
    q, k, pos, (qw, kw) = _inputs(T, H, Hkv, d, BF16)
    inv = _freq(d)
    want = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    rows = torch.full((T, (H + Hkv) * d + 24), float("nan"), dtype=BF16, device="cuda")  # one buffer for both
    qo, ko = rows[:, :H * d].view(T, H, d), rows[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
    q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert rows[:, -24:].isnan().all()
    base = q._base.clone() if q._base is not None else None
    x = torch.cat((q.flatten(1), k.flatten(1), torch.full((T, 40), 7.0, dtype=BF16, device="cuda")), 1)
    q2, k2 = x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
    got = q8.q8_qk_norm_rope(q2, k2, pos, inv, q_weight=qw, k_weight=kw, q_out=q2, k_out=k2)
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1]) and (x[:, -40:] == 7).all()
    assert base is None or torch.equal(base, q._base)  # the inputs of the first call are untouched


def test_one_token_repeated(q8):
    """Stride 0: every position of the same token."""
    q, k, _, (qw, kw) = _inputs(1, 3, 1, 64, F32)
    q, k = q.expand(100, 3, 64), k.expand(100, 1, 64)
    pos, inv = torch.arange(100, device="cuda", dtype=torch.int32), _freq(64)
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    _check(qo, q, pos, inv, qw)
    _check(ko, k, pos, inv, kw)


def test_nan_stays_in_its_head(q8):
    q, k, pos, (qw, kw) = _inputs(5, 4, 2, 128, F32)
    inv = _freq(128)
    want = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    q = q.clone()
    q[2, 1, 77] = float("nan")
    q[3, 0, 5] = float("inf")
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    keep = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[3, 0] = False
    assert torch.equal(qo[keep], want[0][keep]) and torch.equal(ko, want[1]) and qo[2, 1].isnan().all()


def test_empty(q8):
    z = torch.empty(0, 4, 64, device="cuda")
    qo, ko = q8.q8_qk_norm_rope(z, z[:, :2], torch.empty(0, dtype=torch.int32, device="cuda"), _freq(64))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)


def test_rows_behind_4_gigabytes(q8):
    """Tokens 2^27 elements apart: offsets beyond 32 bits, in elements and in bytes."""
    T, d = 40, 64
    try:
        big = torch.empty((T - 1) * (1 << 27) + 256, dtype=BF16, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs 10 GB")
    q, k = big.as_strided((T, 2, d), (1 << 27, d, 1)), big.as_strided((T, 1, d), (1 << 27, d, 1), 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    q.copy_(torch.randn(T, 2, d, generator=g, device="cuda"))
    k.copy_(torch.randn(T, 1, d, generator=g, device="cuda"))
    pos, inv = torch.arange(T, device="cuda", dtype=torch.int32), _freq(d)
    want = q8.q8_qk_norm_rope(q.contiguous(), k.contiguous(), pos, inv)
    q8.q8_qk_norm_rope(q, k, pos, inv, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_refusals(q8):
    q, k, pos, (qw, kw) = _inputs(4, 4, 2, 64, BF16)
    inv = _freq(64)
    with pytest.raises(TypeError, match="k"):
        q8.q8_qk_norm_rope(q, k.float(), pos, inv)
    with pytest.raises(TypeError, match="positions"):
        q8.q8_qk_norm_rope(q, k, pos.long(), inv)
    with pytest.raises(TypeError, match="inv_freq"):
        q8.q8_qk_norm_rope(q, k, pos, inv.float())
    with pytest.raises(ValueError, match="positions"):
        q8.q8_qk_norm_rope(q, k, pos[:3], inv)
    with pytest.raises(ValueError, match="heads of a token"):
        q8.q8_qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, inv)
    with pytest.raises(ValueError, match="channels"):
        q8.q8_qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, inv)
    with pytest.raises(q8.Q8Error, match="Q8_ERR_SHAPE"):
        q8.q8_qk_norm_rope(q, k, pos, inv[:12])            # 24 channels
    with pytest.raises(q8.Q8Error, match="Q8_ERR_SHAPE"):
        q8.q8_qk_norm_rope(q, k, pos, _freq(128))           # more channels than a head has
    with pytest.raises(q8.Q8Error, match="Q8_ERR_VALUE"):
        q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, eps=0.0)
    x = torch.empty(4, 4 * 64 + 4, dtype=BF16, device="cuda")
    with pytest.raises(q8.Q8Error, match="Q8_ERR_ALIGN"):
        q8.q8_qk_norm_rope(x[:, 4:].view(4, 4, 64), k, pos, inv)


def test_captured_and_replayed_and_on_another_stream(q8):
    q, k, pos, (qw, kw) = _inputs(9, 6, 2, 128, BF16)
    inv = _freq(128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qo, ko = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, stream=side)
    side.synchronize()
    _check(qo, q, pos, inv, qw, what="q")
    _check(ko, k, pos, inv, kw, what="k")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        go = q8.q8_qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    for far in (0, 5, 123456):
        pos.copy_(torch.arange(9, dtype=torch.int32) + far)
        g.replay()
        torch.cuda.synchronize()
        _check(go[0], q, pos, inv, qw, what=f"q {far}")
        _check(go[1], k, pos, inv, kw, what=f"k {far}")
