"""The angles of q8_qk_norm_rope: frequencies that have none."""
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
