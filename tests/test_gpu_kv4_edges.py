"""Attention over the 4-bit cache at the limits of its numbers: scores of any size, values near the
largest, what is not finite in parts of a request."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import attention_ref as R  # noqa: E402
from tests import kv4_ref as K  # noqa: E402
from tests.test_gpu_kv4 import BF16, cum, expected, i32, make, q8, queries, widened  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def loud(lens, page, Hkv, d, kexp, sign):
    """make(), with keys of one sign: (1 .. 7) 2^kexp."""
    cache, bt, kv = make(lens, page, Hkv, d, seed=11)
    kc, vc, ks, vs = K.unpack(cache.reshape(-1, 36 * d))
    kc = 8 + sign * (kc - 8).abs().clamp(min=1)
    ks = torch.where(ks.isnan(), ks, torch.full_like(ks, 2.0 ** kexp))
    cache = K.pack(kc, vc, ks, vs).view(cache.shape).cuda()
    return cache, bt, [(sign * (k / s.float().repeat_interleave(32, -1)).abs().clamp(min=1) * 2.0 ** kexp, v, s, vs) for k, v, s, vs in kv]


# scores of 2^17 and more apart, up to the largest that the operands' types allow
SIZES = [(20, 3, 1), (20, 3, -1), (40, 0, 1), (89, -60, -1), (89, 8, -1), (89, 8, 1), (60, 60, -1), (89, 120, 1), (89, 120, -1), (-30, 70, -1)]


@pytest.mark.parametrize("qexp,kexp,sign", SIZES)
@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (4, 4, 64), (16, 4, 256), (24, 2, 128), (32, 2, 64)])
@pytest.mark.parametrize("lens,news,wide", [([1, 0, 300, 45], None, False), ([1, 0, 300, 45], None, True), ([33, 2, 200], [4, 3, 1], False),
                                            ([6000], [2], False), ([6000, 70], None, True)])
def test_scores_of_any_size(q8, lens, news, wide, H, Hkv, d, qexp, kexp, sign):  # noqa: F811
    """Each query has one channel that is not 0, so its scores are exact and equal or far apart: its output is the
    mean of the values of its best keys, however large, or negative, their score is."""
    cache, bt, kv = loud(lens, 64, Hkv, d, kexp, sign)
    cu = cum(news) if news else list(range(len(lens) + 1))
    q = torch.zeros(cu[-1], H, d, device="cuda", dtype=BF16)
    channel = (37 * torch.arange(H, device="cuda")) % d
    q[:, torch.arange(H, device="cuda"), channel] = 1.5 * 2.0 ** qexp
    got = q8.q8_kv4_attention(q, cache, widened(bt) if wide else bt, i32(lens), cu_q=i32(cu) if news else None)
    assert q8.q8_device_error() == 0
    ref, tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for (k, v, _, vs), a, b in zip(kv, cu, cu[1:]):
        n = k.shape[0]
        for i in range(a, b):
            m = n - (b - a) + i - a + 1  # the keys that it sees
            if m <= 0:
                continue
            for h in range(H):
                at = k[:m, h // (H // Hkv), channel[h]]
                best = at == at.max()
                vb, sb = v[:m, h // (H // Hkv)][best].double(), vs[:m, h // (H // Hkv)][best].double().repeat_interleave(32, -1)
                ref[i, h] = vb.mean(0)
                # as in kv4_ref, with exact scores
                tol[i, h] = K.STEP * (vb.abs().mean(0) + ref[i, h].abs()) * (1 + 2.0 ** -5) + (m + 64) * 2.0 ** -22 * 25.0 * sb.mean(0)
    R.assert_within(got, ref, tol, "loud scores")


@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (4, 4, 64), (16, 4, 256), (24, 2, 128), (32, 2, 64)])
@pytest.mark.parametrize("lens,news,wide", [([1, 0, 300, 45], None, False), ([33, 2, 200], [4, 3, 1], False), ([6000, 70], None, True)])
def test_values_near_the_largest(q8, lens, news, wide, H, Hkv, d):  # noqa: F811
    """Values up to 2^50, queries just below 2^90 with scores of the usual size."""
    cache, bt, kv = make(lens, 64, Hkv, d, seed=12)
    scales = cache.view(-1, 36 * d)[:, 34 * d:].view(BF16)
    scales *= 2.0 ** 47
    kv = [(k, v * 2.0 ** 47, ks, vs * 2.0 ** 47) for k, v, ks, vs in kv]
    cu = cum(news) if news else list(range(len(lens) + 1))
    q = queries(cu[-1], H, d)
    q = (q.float() * (0.99 * 2.0 ** 90 / q.float().abs().amax().item() if q.numel() else 1.0)).to(BF16)
    scale = 2.0 ** -88 * d ** -0.5
    got = q8.q8_kv4_attention(q, cache, widened(bt) if wide else bt, i32(lens), cu_q=i32(cu) if news else None, scale=scale)
    assert q8.q8_device_error() == 0
    assert max(float(v.abs().max()) for _, v, _, _ in kv if v.numel()) > 2.0 ** 47
    R.assert_within(got, *expected(q, kv, cu, scale), "large values")


@pytest.mark.parametrize("odd", [math.nan, math.inf])
@pytest.mark.parametrize("Hkv,d,tokens,news", [(1, 128, 19200, [1]), (2, 64, 20000, [1]), (2, 256, 12000, [2]), (1, 128, 40000, None)])
def test_a_value_among_keys_that_count_for_nothing(q8, Hkv, d, tokens, news, odd):  # noqa: F811
    """A value that is not finite, in a stretch of keys whose score is -infinity (weight 0) that takes up whole
    blocks' parts of the request: its rows are NaN all the same, 0 times it."""
    H = 4 * Hkv
    cache, bt, _ = make([tokens], 64, Hkv, d, seed=13)
    if news is None:
        bt = widened(bt)
    kc, vc, ks, vs = K.unpack(cache.reshape(-1, 36 * d))
    n = 64 // 32
    q = queries(sum(news or [1]), H, d)
    q[..., :32] = 0
    q[..., 5] = 1.0            # the first block's scores are its codes times its scale
    at = torch.arange(tokens // 4, tokens * 3 // 4)
    tile = (bt[0].cpu()[at // 64].long() * Hkv) * n + at % 64 // 32   # of head 0
    kc[tile, at % 32, 5] = 1   # -7
    ks[tile, at % 32, 0] = math.inf
    mid = len(at) // 2
    vs[tile[mid], at[mid] % 32, 1] = odd
    cache = K.pack(kc, vc, ks, vs).view(cache.shape).cuda()
    got = q8.q8_kv4_attention(q, cache, bt, i32([tokens]), cu_q=i32(cum(news)) if news else None)
    assert q8.q8_device_error() == 0
    assert got[:, :4].isnan().all()
    assert got[:, 4:].isfinite().all()
