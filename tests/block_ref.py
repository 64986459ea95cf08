"""LayerNorm, rotary positions and the head RMSNorm with rotary positions in 64
bits, as plainly as their definitions, with bounds on the fp32 kernels' errors.

u = 2^-24 is half a step of fp32, one rounding's relative error. K = 96 bounds
the additions on one path of a row's sum: at most 64 values a thread, 5 steps of
a warp's butterfly, at most 16 warps' totals, and slack. Every
bound below is a sum of |term| * (roundings on the term's way) * u; an output in
16 bits adds half a step of its format at the larger of the two values compared.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
K = 96
RSQRT = 2.0 ** -22  # rsqrtf: 2 ulp


def half_step(v: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Half the spacing of ``dtype`` at |v| (float64 in, float64 out), subnormals included."""
    bits, emin = (7, -126) if dtype == torch.bfloat16 else (10, -14)
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** emin)))
    return torch.exp2(e - bits - 1)


def assert_within(name, got, ref, bound, dtype=None):
    """|got - ref| <= bound (+ half a step of ``dtype``), element by element."""
    got = got.double()
    lim = bound if dtype is None else bound + half_step(torch.maximum(got.abs(), ref.abs()), dtype)
    bad = ~((got - ref).abs() <= lim)  # a NaN is bad
    if bool(bad.any()):
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got[i])!r}, "
                             f"want {float(ref[i])!r} within {float(lim[i]):.3g}")


def effective(w, zc):
    return ((w + 1.0) if zc else w).double()  # the +1 is an fp32 addition


# --------------------------------------------------------------------------
# LayerNorm
# --------------------------------------------------------------------------
def ln_fwd(x, w, b, eps):
    """(y, mean, rstd) and their bounds, from float64 x [T, D]."""
    D = x.shape[1]
    mean = x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = (var + eps) ** -0.5
    n = c * rstd[:, None]
    y = n * w + (0.0 if b is None else b)
    e_mean = (K + 1) * U * x.abs().mean(1)
    # sum of (c + d)^2 = sum c^2 + D d^2: the mean's error d enters squared
    e_r = 0.5 * ((K + 4) * U + e_mean ** 2 / (var + eps)) + RSQRT
    e_y = (w * rstd[:, None]).abs() * e_mean[:, None] + (n * w).abs() * (e_r[:, None] + 5 * U) + U * y.abs()
    return (y, mean, rstd), (e_y, e_mean, rstd * e_r)


def ln_bwd(g, x, w, mean, rstd):
    """(dx, dw, db) and their bounds, from the float64 inputs and the saved statistics."""
    T, D = x.shape
    n = (x - mean[:, None]) * rstd[:, None]
    gw = g * w
    c1 = gw.mean(1, keepdim=True)
    c2 = (gw * n).mean(1, keepdim=True)
    dx = rstd[:, None] * (gw - c1 - n * c2)
    size = gw.abs() + gw.abs().mean(1, keepdim=True) + n.abs() * (gw * n).abs().mean(1, keepdim=True)
    e_dx = (K + 8) * U * rstd[:, None].abs() * size
    chain = rows_chain(T)
    return (dx, (g * n).sum(0), g.sum(0)), (e_dx, (chain + 4) * U * (g * n).abs().sum(0), chain * U * g.abs().sum(0))


def rows_chain(T):
    """Additions on one path of a weight gradient's sum over T rows, at the sizes that
    are checked with it: a lane's rows and its CTA's groups (together at most 256
    there), 16 and 8 of the ranges' totals, the chunks of one range, slack. The tests
    of longer sums, of 256 rows and more a lane, count their chains themselves."""
    return min(T, 256) + 32 + T // 2048 + 8


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
def turned(x, pos, inv_freq, scale, interleaved, back=False):
    """x [T, H, D] (float64) with its first 2 * len(inv_freq) values a head turned, and, beside it, scale
    times |u| + |v| of each value's pair (0 where nothing is turned)."""
    R = 2 * inv_freq.shape[0]
    a = pos.double()[:, None, None] * inv_freq
    c, s = a.cos() * scale, a.sin() * scale
    if back:
        s = -s
    out, size = x.clone(), torch.zeros_like(x)
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    u, v = x[..., i], x[..., j]
    out[..., i] = u * c - v * s
    out[..., j] = v * c + u * s
    size[..., i] = size[..., j] = abs(scale) * (u.abs() + v.abs())
    return out, size


# A turned value's error over scale * (|u| + |v|), in u: the angle, 1.6 (below a
# quarter turn it is rounded twice as fp32; the phase's 2^-55 turns and the
# frequency's |a| 2^-51 are far less here); the series of sine and cosine, 1.5; the
# scale, 1; a product and a fused sum, 2. Together under 8.
TURN = 8 * U


def norm_turn_fwd(x, w, eps, pos, inv_freq, scale, interleaved):
    """(out, rstd) and their bounds, from float64 x [T, H, D]."""
    rstd = ((x * x).mean(2) + eps) ** -0.5
    e_r = 0.5 * (K + 3) * U + RSQRT
    n = x * rstd[..., None] * w
    out, size = turned(n, pos, inv_freq, scale, interleaved)
    turn = 2 * inv_freq.shape[0]
    size[..., turn:] = n[..., turn:].abs()
    return (out, rstd), (size * (e_r + 3 * U + TURN), rstd * e_r)


def norm_turn_bwd(g, x, w, rstd, pos, inv_freq, scale, interleaved):
    """(dx, dw) and their bounds."""
    T, H, D = x.shape
    r = rstd[..., None]
    gt, size = turned(g, pos, inv_freq, scale, interleaved, back=True)
    e_g = TURN * size
    dot = (gt * w * x).sum(2, keepdim=True)
    dx = gt * w * r - x * (r ** 3 / D) * dot
    e_dot = ((w * x).abs() * e_g).sum(2, keepdim=True) + (K + 4) * U * (gt * w * x).abs().sum(2, keepdim=True)
    e_dx = (w * r).abs() * e_g + 4 * U * (gt * w * r).abs() + (x * r ** 3 / D).abs() * (e_dot + 6 * U * dot.abs())
    n = x * r
    e_dw = (n.abs() * e_g).sum((0, 1)) + (rows_chain(T * H) + 4) * U * (gt * n).abs().sum((0, 1))
    return (dx, (gt * n).sum((0, 1))), (e_dx, e_dw)
