"""The angles of q8_qk_norm_rope: how exact they are, and frequencies that have none.

A pair (a, b) = (sin t, cos t) in binary32 turns to (a cos t - b sin t, ...): its first channel is
almost 0, so that the rounding of the output to bfloat16 is too, and an angle that is off shows in
full.  The angle may be off by 2^-25 turns, sine and cosine by one unit in the last place (2^-24)
each, the two products and their difference by 2^-25 of |a| + |b| each:
    |out - ref| <= 2^-8 |ref| (1 + 2^-7) + (|a| + |b|) (2 pi 2^-25 + 2^-23).
The products position * frequency are exact in binary64: frequencies of at most 21 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as m
    torch.cuda.set_device(0)
    return m


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [100, 1 << 20, (1 << 31) - 1])
def test_angles_to_the_stated_bound(q8, top, interleaved):
    T, half = 2000, 128
    g = torch.Generator(device="cuda").manual_seed(top & 0xFFFF)
    pos = torch.randint(-top, top, (T,), generator=g, device="cuda").int()
    pos[0], pos[1] = top, -top
    inv = torch.randint(0, (1 << 21) + 1, (half,), generator=g, device="cuda").double() * 2.0 ** -21
    inv[0], inv[1], inv[2] = 1.0, -1.0, 2.0 ** -21
    t = pos.double()[:, None] * inv
    a, b = t.sin().float(), t.cos().float()
    x = torch.stack((a, b), -1).flatten(1) if interleaved else torch.cat((a, b), 1)
    q = x.view(T, 1, 2 * half)
    qo, ko = q8.q8_qk_norm_rope(q, q[:, :0], pos, inv, interleaved=interleaved)
    y = qo.view(T, half, 2) if interleaved else qo.view(T, 2, half).transpose(1, 2)
    a, b = a.double(), b.double()
    ref = torch.stack((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), -1)
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -7) + (a.abs() + b.abs())[..., None] * (2 * math.pi * 2.0 ** -25 + 2.0 ** -23)
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())
    assert ko.shape == (T, 0, 2 * half) and q8.q8_device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan, 2.0 ** 32, -2.0 ** 32, 1e30, -1e300])
def test_a_frequency_without_an_angle_makes_nan_of_its_pairs(q8, bad, interleaved):
    inv = torch.tensor([0.5, bad, 0.25, 0.0, 1.0, 3.0, 2.0 ** 31, 0.125], device="cuda", dtype=torch.float64)
    fine = inv.clone()
    fine[1] = 0.0
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(7, 2, 48, generator=g, device="cuda")
    pos = torch.arange(7, device="cuda", dtype=torch.int32)
    w = torch.ones(48, device="cuda")
    out = q8.q8_qk_norm_rope(q, q[:, :1], pos, inv, q_weight=w, interleaved=interleaved)
    want = q8.q8_qk_norm_rope(q, q[:, :1], pos, fine, q_weight=w, interleaved=interleaved)
    pair = [2, 3] if interleaved else [1, 9]
    rest = [c for c in range(48) if c not in pair]
    for x, y in zip(out, want):
        assert x[..., pair].isnan().all()
        assert torch.equal(x[..., rest], y[..., rest]) and y.isfinite().all()
    assert q8.q8_device_error() == 0
