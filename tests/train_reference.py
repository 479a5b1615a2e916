"""The training operators in 64 bits, from their definitions, and the bounds
their kernels are held to (tests only).

Every function returns (value, magnitude) pairs: the value in fp64 and, for the
bound, the sum of the absolute values of the terms that make it up.  A kernel's
result may differ by half a step of its type from the exact value, plus
`depth` fp32 roundings (2^-24 each) of that magnitude, where depth counts the
operations on the longest path to an output: see `check`.
"""
import math

import torch

F64 = torch.float64
U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def check(got, want, depth, what):
    value, mag = want
    assert tuple(got.shape) == tuple(value.shape), f"{what}: shape {tuple(got.shape)}"
    if got.numel() == 0:
        return
    g = got.to(F64)
    assert torch.isfinite(g).all(), f"{what}: non-finite"
    err = (g - value).abs()
    # a result that rounds to the type from within the fp32 error: both add up
    fp32 = depth * U32 * mag
    tol = HALF_STEP[got.dtype] * (value.abs() + fp32) + fp32 + 1e-37
    bad = err > tol
    if bad.any():
        i = int((err / tol).argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {err.numel()} out of bound; worst {float(err.flatten()[i]):.3e}"
            f" against {float(tol.flatten()[i]):.3e} (value {float(value.flatten()[i]):.6e})")


def key_of_rows(B, L, n_video, device):
    r = torch.arange(L, device=device)
    return 2 * torch.arange(B, device=device)[:, None] + (r >= n_video).long()[None]


def spread(vec, n_video, L):
    """[B, 2, D] vectors over the rows [B, L, D]."""
    B, _, D = vec.shape
    return vec.to(F64).reshape(2 * B, D)[key_of_rows(B, L, n_video, vec.device)]


def key_sums(t, n_video):
    B, L, D = t.shape
    out = torch.zeros((2 * B, D), dtype=F64, device=t.device)
    out.index_add_(0, key_of_rows(B, L, n_video, t.device).reshape(-1), t.reshape(-1, D))
    return out.view(B, 2, D)


def layer_norm(x, gamma, beta, scale, shift, n_video, eps):
    B, L, D = x.shape
    x = x.to(F64)
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    g = torch.ones(D, dtype=F64, device=x.device) if gamma is None else gamma.to(F64)
    b = torch.zeros(D, dtype=F64, device=x.device) if beta is None else beta.to(F64)
    sc = spread(scale, n_video, L) if scale is not None else torch.zeros_like(x)
    sh = spread(shift, n_video, L) if shift is not None else torch.zeros_like(x)
    y = (xc * rstd * g + b) * (1 + sc) + sh
    absmean = x.abs().mean(-1, keepdim=True)
    mag = ((x.abs() + absmean) * rstd * g.abs() + b.abs()) * (1 + sc.abs()) + sh.abs()
    # rstd's own relative error grows with the rounding of x - mean
    spread_err = rstd * (x.abs() + absmean).square().mean(-1, keepdim=True).sqrt()
    return ((y, mag * (1 + spread_err)), (mean[..., 0], absmean[..., 0]),
            (rstd[..., 0], (rstd * (1 + spread_err))[..., 0]))


def norm_backward(dy, x, mean, rstd, gamma, beta, scale, dres, n_video, eps, rms):
    """Returns dict of (value, magnitude): dx, dgamma, dbeta, dscale, dshift."""
    B, L, D = x.shape
    x, dy = x.to(F64), dy.to(F64)
    one = torch.ones(D, dtype=F64, device=x.device)
    g = one if gamma is None else gamma.to(F64)
    b = torch.zeros_like(one) if beta is None else beta.to(F64)
    fac = 1 + spread(scale, n_video, L) if scale is not None else torch.ones_like(x)
    if rms:
        rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        xc = x
        xa = x.abs()
    else:
        rs = rstd.to(F64)[..., None]
        xc = x - mean.to(F64)[..., None]
        xa = x.abs() + mean.to(F64).abs()[..., None]     # what xc's rounding is relative to
    xh, xha = xc * rs, xa * rs
    gg, ga = dy * fac * g, (dy * fac * g).abs()
    m1 = torch.zeros_like(rs) if rms else gg.mean(-1, keepdim=True)
    m1a = torch.zeros_like(rs) if rms else ga.mean(-1, keepdim=True)
    m2 = (gg * xh).mean(-1, keepdim=True)
    m2a = (ga * xha).mean(-1, keepdim=True)
    dx = rs * (gg - m1 - xh * m2)
    dxa = rs * (ga + m1a + xha * m2a)
    if dres is not None:
        dx = dx + dres.to(F64)
        dxa = dxa + dres.to(F64).abs()
    dfac = dy * fac
    n, na = xh * g + b, xha * g.abs() + b.abs()
    return {
        "dx": (dx, dxa),
        "dgamma": ((dfac * xh).sum((0, 1)), (dfac.abs() * xha).sum((0, 1))),
        "dbeta": (dfac.sum((0, 1)), dfac.abs().sum((0, 1))),
        "dscale": (key_sums(dy * n, n_video), key_sums(dy.abs() * na, n_video)),
        "dshift": (key_sums(dy, n_video), key_sums(dy.abs(), n_video)),
    }


def philox(counter, key, rounds=10):
    """Philox4x32 on python integers: four 32-bit counter words, two key words."""
    m = 0xFFFFFFFF
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & m, (p0 >> 32) ^ c[3] ^ k[1], p0 & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def keep_mask(n, seed, offset, p, device, first=0):
    """keep of elements first .. first + n of a tensor, from 64-bit torch
    integers (products split so that none passes 2^63)."""
    m = 0xFFFFFFFF
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    lo = first // 4
    i = torch.arange(lo, (first + n + 3) // 4, device=device)

    def mul(x, c):
        a, b = x * (c & 0xFFFF), x * (c >> 16)
        s = a + ((b & 0xFFFF) << 16)
        return (b >> 16) + (s >> 32), s & m

    c = [i & m, i >> 32, torch.full_like(i, offset & m), torch.full_like(i, offset >> 32)]
    k = [seed & m, seed >> 32]
    for _ in range(10):
        h0, l0 = mul(c[0], 0xD2511F53)
        h1, l1 = mul(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    words = torch.stack(c, 1).reshape(-1)[first - 4 * lo:first - 4 * lo + n]
    return words >= round(p * 2.0 ** 32)


def p32(p):
    return torch.tensor(p, dtype=torch.float32).item()


def dropped(t, rng, site, p):
    """keep * t / (1 - p), 0 where dropped."""
    seed, offset = rng
    p = p32(p)
    keep = keep_mask(t.numel(), seed, offset + site, p, t.device).view(t.shape)
    k = 1.0 / (1.0 - p) if p < 1 else 0.0
    return torch.where(keep, t.to(F64) * k, torch.zeros((), dtype=F64, device=t.device))


def pair_map(sections, theta, per_axis, interleaved):
    """(axis, frequency) of every pair, from the words of the definition."""
    n, P = len(sections), sum(sections)
    if interleaved:
        order = [(a, j) for j in range(max(sections)) for a in range(n) if j < sections[a]]
    else:
        order = [(a, j) for a in range(n) for j in range(sections[a])]
    return [(a, theta ** (-(j / sections[a]) if per_axis else -i / P))
            for i, (a, j) in enumerate(order)]


def rotate(t, pos, pairs, half, sign=1.0):
    """t [B, L, H, hd] fp64 at pos [n_axes, B, L], every pair as a 2 x 2 matrix."""
    P = len(pairs)
    out, mag = t.clone(), t.abs().clone()
    pos = pos.to(F64)
    for i, (a, f) in enumerate(pairs):
        u, v = (i, i + P) if half else (2 * i, 2 * i + 1)
        phi = sign * pos[a] * f
        c, s = torch.cos(phi)[..., None], torch.sin(phi)[..., None]
        out[..., u] = t[..., u] * c - t[..., v] * s
        out[..., v] = t[..., u] * s + t[..., v] * c
        mag[..., u] = mag[..., v] = t[..., u].abs() + t[..., v].abs()
    return out, mag


def rope(x, pos, pairs, half, norm, gamma, eps):
    x = x.to(F64)
    if norm:
        rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        x = x * rs * (1.0 if gamma is None else gamma.to(F64))
    return rotate(x, pos, pairs, half)


def rope_backward(dy, x, pos, pairs, half, norm, gamma, eps):
    """((dx, mag), (dgamma, mag) or None)."""
    g, ga = rotate(dy.to(F64), pos, pairs, half, -1.0)
    if not norm:
        return (g, ga), None
    x = x.to(F64)
    rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * rs
    w = torch.ones(x.shape[-1], dtype=F64, device=x.device) if gamma is None else gamma.to(F64)
    gg, gga = g * w, ga * w.abs()
    dx = rs * (gg - xh * (gg * xh).mean(-1, keepdim=True))
    dxa = rs * (gga + xh.abs() * (gga * xh.abs()).mean(-1, keepdim=True))
    return (dx, dxa), ((g * xh).sum((0, 1, 2)), (ga * xh.abs()).sum((0, 1, 2)))


def depth_row(D):
    """Roundings on the path through a row's sum: a thread adds at most 64 of
    the row's products in its lane, a warp joins 32 lanes, a CTA at most 16
    warps; about 16 more operations make the result from the sums."""
    return 64 + 5 + 16 + 16


def depth_rows(rows):
    """... through a sum over rows, each term a product of a few factors: in
    the worst case one thread adds every row."""
    return rows + 32


def assert_derivative(f, x, direction, claimed, h=1e-6, rel=1e-6):
    """The derivative of the fp64 scalar f at x along `direction` from central
    differences, against the one claimed."""
    d = (f(x + h * direction) - f(x - h * direction)) / (2 * h)
    assert math.isclose(float(d), float(claimed), rel_tol=rel, abs_tol=rel), (float(d),
                                                                               float(claimed))
