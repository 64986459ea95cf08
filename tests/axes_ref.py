"""Rotary positions of several axes and the head norm with them in 64 bits, with the
bounds of ``tests/block_ref.py`` (a pair's arithmetic is that of one axis)."""
from __future__ import annotations

import torch

from tests.block_ref import K, RSQRT, TURN, U, rows_chain


def turned(x, pos, axis, inv_freq, scale, interleaved, back=False):
    """x [T, H, D] (float64), pos [axes, T] and the pairs' axes: the turned heads and scale times |u| + |v| of each
    value's pair (0 where nothing is turned)."""
    n = inv_freq.shape[0]
    angle = torch.stack([pos[int(axis[i])].double() * inv_freq[i] for i in range(n)], 1)[:, None]
    z = torch.polar(torch.full_like(angle, scale), -angle if back else angle)
    i = torch.arange(n, device=x.device)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    out, size = x.clone(), torch.zeros_like(x)
    w = torch.complex(x[..., u], x[..., v]) * z
    out[..., u], out[..., v] = w.real, w.imag
    size[..., u] = size[..., v] = abs(scale) * (x[..., u].abs() + x[..., v].abs())
    return out, size


def norm_turn_fwd(x, w, eps, pos, axis, inv_freq, scale, interleaved):
    rstd = ((x * x).mean(2) + eps) ** -0.5
    e_r = 0.5 * (K + 3) * U + RSQRT
    n = x * rstd[..., None] * w
    out, size = turned(n, pos, axis, inv_freq, scale, interleaved)
    rest = 2 * inv_freq.shape[0]
    size[..., rest:] = n[..., rest:].abs()
    return (out, rstd), (size * (e_r + 3 * U + TURN), rstd * e_r)


def norm_turn_bwd(g, x, w, rstd, pos, axis, inv_freq, scale, interleaved):
    T, H, D = x.shape
    r = rstd[..., None]
    gt, size = turned(g, pos, axis, inv_freq, scale, interleaved, back=True)
    e_g = TURN * size
    dot = (gt * w * x).sum(2, keepdim=True)
    dx = gt * w * r - x * (r ** 3 / D) * dot
    e_dot = ((w * x).abs() * e_g).sum(2, keepdim=True) + (K + 4) * U * (gt * w * x).abs().sum(2, keepdim=True)
    e_dx = (w * r).abs() * e_g + 4 * U * (gt * w * r).abs() + (x * r ** 3 / D).abs() * (e_dot + 6 * U * dot.abs())
    n = x * r
    e_dw = (n.abs() * e_g).sum((0, 1)) + (rows_chain(T * H) + 4) * U * (gt * n).abs().sum((0, 1))
    return (dx, (gt * n).sum((0, 1))), (e_dx, e_dw)
