"""Plain forms of the paged 4-bit cache's operators, and the error their kernels may make.

A tile of 32 tokens, byte by byte (index arrays from loops over the format's definition), the
quantiser in binary32 with one rounding per operation, and attention in binary64.

Attention.  The product of a weight p_j and a value's scale is rounded to bfloat16 (half a step, 2^-8
relative; the weight's own leading bits and rest leave 2^-14 of it beside that), and o once: with A =
sum p_j |v_j| / sum p_j that is below 2^-8 (A + |ref|) (1 + 2^-5).  In binary32 the kernel sums nibbles n = code + 8 in 1 .. 15 (for outputs every other
one as (n + 16 n' less n) / 16) and takes 8 times the other factor's sum off: terms of up to 15 + 8,
or (255 + 15) / 16 + 8, both below 25, times |q_i| s for a score, p_j s for an output, instead of
|q_i k_i| and p_j |v_j|.  So a score is off by at most (d + 8) 2^-23 scale 25 sum_i |q_i| s =: g
(the tensor pipe may cut sums off instead of rounding them, hence 2^-23), which takes every weight,
and so their sum, to between e^-g and e^g times itself: p_j / sum p stays within a factor e^(2 g),
and o moves by at most (e^(2 g) - 1) A; sums of n weights, the exponential (its argument, up to
2^7, rounded to 2^-17) and the division add (n + 64) 2^-22 of A' = 25 sum p_j s / sum p_j.
    |o - ref| <= 2^-8 (A + |ref|) (1 + 2^-5) + (e^(2 g) - 1) A + (n + 64) 2^-22 A'.
"""
import torch

STEP = 2.0 ** -8


def places(d):
    """(key bytes, key shifts, value bytes, value shifts) of the codes [32 tokens, d channels] in a tile."""
    kb, ks, vb, vs = ([[0] * d for _ in range(32)] for _ in range(4))
    quads, words, halves = max(1, d // 128), min(4, d // 32), d // 64
    for t in range(4):
        for j in range(4):
            for i in range(2):
                tok = 8 * t + 2 * j + i
                for c in range(d):
                    b, u, nib = c // 32, c % 32 // 8, c % 8
                    word = (((j * quads + b // 4) * 8 + (2 * t + i)) * 4 + u) * words + b % 4
                    kb[tok][c], ks[tok][c] = 4 * word + nib // 2, 4 * (nib % 2)
                    h, low, g = c // 64, c % 64 < 32, c % 32 // 4
                    nib = c % 4 + (0 if low else 4)
                    word = (((2 * j + i) * 8 + g) * 4 + t) * halves + h
                    vb[tok][c], vs[tok][c] = 18 * d + 4 * word + nib // 2, 4 * (nib % 2)
    return tuple(torch.tensor(x) for x in (kb, ks, vb, vs))


def pack(kc, vc, ksc, vsc):
    """Codes int [n, 32, d] in 0 .. 15 and scales bfloat16 [n, 32, d / 32] -> tiles uint8 [n, 36 d]."""
    n, _, d = kc.shape
    kb, ks, vb, vs = places(d)
    out = torch.zeros(n, 36 * d, dtype=torch.int32)
    for codes, at, sh in ((kc, kb, ks), (vc, vb, vs)):
        out.index_add_(1, at.flatten(), (codes.cpu().int() << sh.int()).view(n, -1).int())
    out = out.to(torch.uint8)
    for sc, at in ((ksc, 16 * d), (vsc, 34 * d)):
        out[:, at:at + 2 * d] = sc.cpu().transpose(1, 2).contiguous().view(torch.uint8).view(n, -1)
    return out


def unpack(tiles):
    """Tiles uint8 [n, 36 d] -> (key codes, value codes) int [n, 32, d], (key, value) scales [n, 32, d / 32]."""
    tiles = tiles.cpu()
    n, d = tiles.shape[0], tiles.shape[1] // 36
    kb, ks, vb, vs = places(d)
    codes = [(tiles[:, at.flatten()].int().view(n, 32, d) >> sh) & 15 for at, sh in ((kb, ks), (vb, vs))]
    scales = [tiles[:, at:at + 2 * d].contiguous().view(torch.bfloat16).view(n, d // 32, 32).transpose(1, 2) for at in (16 * d, 34 * d)]
    return codes[0], codes[1], scales[0], scales[1]


def values(codes, scales):
    """What codes [n, 32, d] and scales [n, 32, d / 32] stand for, binary32 (exact)."""
    return (codes.float() - 8.0) * scales.float().repeat_interleave(32, -1)


def turned(x, w, table, interleaved):
    """[T, heads, d] float32: x * w with its first pairs turned, one rounding per operation (CPU)."""
    z = x.float()
    z = z if w is None else z * w
    if table is None:
        return z
    half = table.shape[2]
    cos, sin = table[:, 0, None], table[:, 1, None]
    out = z.clone()
    a, b = (z[..., 0:2 * half:2], z[..., 1:2 * half:2]) if interleaved else (z[..., :half], z[..., half:2 * half])
    u, v = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = u, v
    else:
        out[..., :half], out[..., half:2 * half] = u, v
    return out


def quantised(z):
    """float32 [.., d] -> (codes 0 .. 15, largest magnitudes [.., d / 32]); CPU, one rounding per operation."""
    y = z.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    small = top < 2.0 ** -120
    inv = torch.where(small, torch.zeros_like(top), torch.full_like(top, 7.0) / top)
    codes = (y * inv[..., None]).round().int() + 8
    return codes.flatten(-2), torch.where(small, torch.zeros_like(top), top)


def attention(q, k, v, ks, vs, seen, scale):
    """q [n, H, d] bfloat16, k and v [m, Hkv, d] and their scales [m, Hkv, d / 32], seen [n, m] ->
    (o, tolerance) binary64."""
    G = q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    n, d = max(1, k.shape[0]), q.shape[2]
    for h in range(q.shape[1]):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        if not kh.shape[0] or not qh.shape[0]:
            continue
        sk, sv = (x[:, h // G].double().repeat_interleave(32, -1) for x in (ks, vs))
        x = (qh @ kh.T * scale).masked_fill(~seen, -torch.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top.masked_fill(top == -torch.inf, 0.0))
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
        g = (d + 8) * 2.0 ** -23 * scale * 25.0 * ((qh.abs() @ sk.T) * seen).amax(-1, keepdim=True)
        a, wide = p @ vh.abs(), 25.0 * (p @ sv)
        o[:, h] = p @ vh
        tol[:, h] = STEP * (a + o[:, h].abs()) * (1 + 2.0 ** -5) + torch.expm1(2 * g) * a + (n + 64) * 2.0 ** -22 * wide
    return o, tol
