"""Plain binary64 forms of the attention layer's operators, and the error their kernels may
make.

Attention.  The kernels round each weight p_j to bfloat16 before the product with v (half a
step, 2^-8 relative) and o once more (2^-8 of its value); A = sum p_j |v_j| / sum p_j bounds
what the first costs.  In binary32: a score is a sum of d exact products, off by at most
(d + 4) 2^-24 scale sum_i |q_i k_i| =: g, which moves a weight and the weights' sum by e^g - 1
each, at most 2.2 g each for g < 0.4; sums of n weights and products, the exponential and the
division add (n + 16) 2^-23.  So
    |o - ref| <= 2^-8 (A + |ref|) (1 + 2^-7) + A (4.4 g + (n + 16) 2^-23).

Rotation.  |z| is off by at most (d / 2 + 8) 2^-24 relative (the sum of squares, its root, two
products): below 2^-16 for d <= 256; the angle by 2^-32 turns and its binary32 rounding, with
sine and cosine below 2^-21; so a pair (a, b) gives
    |out - ref| <= 2^-8 |ref| (1 + 2^-7) + (|a| + |b|) 2^-15.
"""
import torch

STEP = 2.0 ** -8


def _softmax_rows(q, k, v, seen, scale):
    """q [n, H, d], k and v [m, Hkv, d] any float type, seen [n, m] -> (o, tolerance)."""
    G = q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    n, d = max(1, k.shape[0]), q.shape[2]
    for h in range(q.shape[1]):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        if not kh.shape[0] or not qh.shape[0]:
            continue
        x = (qh @ kh.T * scale).masked_fill(~seen, -torch.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top.masked_fill(top == -torch.inf, 0.0))
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
        size = ((qh.abs() @ kh.abs().T) * seen).amax(-1, keepdim=True) * scale
        g = (d + 4) * 2.0 ** -24 * size
        assert float(g.max()) < 0.4
        a = p @ vh.abs()
        o[:, h] = p @ vh
        tol[:, h] = STEP * (a + o[:, h].abs()) * (1 + 2.0 ** -7) + a * (4.4 * g + (n + 16) * 2.0 ** -23)
    return o, tol


def prompt(q, k, v, cu_q, cu_k, scale=None):
    """(o, tolerance) of packed sequences; rows outside them are NaN with tolerance 0."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        seen = torch.ones(b - a, d - c, dtype=torch.bool, device=q.device).tril((d - c) - (b - a))
        o[a:b], tol[a:b] = _softmax_rows(q[a:b], k[c:d], v[c:d], seen, scale)
    return o, tol


def prefix(q, kp, vp, ko, vo, own_len, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for b, n in enumerate(own_len):
        k, v = torch.cat((kp, ko[b, :n])), torch.cat((vp, vo[b, :n]))
        seen = torch.ones(1, k.shape[0], dtype=torch.bool, device=q.device)
        o[b:b + 1], tol[b:b + 1] = _softmax_rows(q[b:b + 1], k, v, seen, scale)
    return o, tol


def norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    """(out, tolerance) for the heads x [T, H, d]."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    rot = 2 * inv_freq.shape[0]
    t = positions.double()[:, None, None] * inv_freq.double()
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    out, size = x.clone(), x.abs()
    out[..., ia], out[..., ib] = a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, STEP * out.abs() * (1 + 2.0 ** -7) + size * 2.0 ** -15


def assert_within(got, ref, tol, what=""):
    """Every element within its tolerance; NaN reference elements have to be NaN."""
    got = got.double()
    bad = ~((got - ref).abs() <= tol) & ~(ref.isnan() & got.isnan())
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements outside the tolerance, first {at}: "
                             f"{float(got[at])} for {float(ref[at])} +- {float(tol[at])}")
