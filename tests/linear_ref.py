"""The projections and the gated block in 64 bits, as plainly as their
definitions, with bounds on the kernels' errors.

A matrix product's bound. Products of 16-bit values are exact in fp32. The tensor
core adds 16 of them to the accumulator at a time: the 17 terms are aligned to the
largest one and cut off at fp32's last place there or finer, 2^-23 of that term's
power of two, so a step is off by at most 17 x 2^-23 x (largest prefix sum + largest
product), and a value by that times its ceil(K / 16) steps.

An activation's bound: (its roundings) x |value|, where the argument of an exponential
or of erfc counts with its own size; a derivative's is taken of the sizes of its two
terms. dz, dgate and dup are rounded to 16 bits before their products: where the fp32 value may lie
on either side of a rounding's border, the products' bound has the step times the other operand.
"""
from __future__ import annotations

import math

import torch

from tests.block_ref import U

C2 = math.sqrt(2.0 / math.pi)


def act(name, z):
    """(value, slope) of float64 z and their bounds."""
    az = z.abs()
    if name == "none":
        return (z, torch.ones_like(z)), (0.0 * z, 0.0 * z)
    if name == "relu":
        return (z.clamp_min(0.0), (z > 0).double()), (0.0 * z, 0.0 * z)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(z * -math.sqrt(0.5))
        d = torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        a, s = z * p, p + z * d
        # erfc(t) answers a relative error of t with 2 t^2 and a little of it: z^2 here, below zero alone
        rel = (16.0 + 4.0 * torch.where(z < 0, z * z, torch.zeros_like(z))) * U
        small = 2.0 ** -120
        return (a, s), (a.abs() * rel + small, p * rel + az * d * (16.0 + 4.0 * z * z) * U + small)
    v = z
    dv = torch.ones_like(z)
    if name == "gelu_tanh":
        v = 2.0 * C2 * (z + 0.044715 * z ** 3)
        dv = 2.0 * C2 * (1.0 + 3.0 * 0.044715 * z * z)
    s, t = torch.sigmoid(v), torch.sigmoid(-v)
    rel = (24.0 + 10.0 * v.abs().clamp_max(400.0)) * U
    small = 2.0 ** -120
    if name == "sigmoid":
        return (s, s * t), (s * torch.where(v > 0, 24.0 * U + 0 * v, rel) + small, s * t * rel + small)
    a = z * s
    rel_a = torch.where(v > 0, 24.0 * U + t * rel, rel)
    both = az * s * t * dv
    slope = s + torch.where(s * t == 0, 0.0 * z, z * s * t * dv)
    both = torch.where(s * t == 0, 0.0 * z, both)
    return (a, slope), (a.abs() * rel_a + az * small, s * rel_a + both * 2.0 * rel + small)


def product(a, b):
    """a [M, K] b [N, K]^T in float64 and its bound."""
    M, K = a.shape
    acc = torch.zeros((M, b.shape[0]), dtype=torch.float64, device=a.device)
    top = torch.zeros_like(acc)
    for k in range(0, K, 16):
        acc = acc + a[:, k:k + 16] @ b[:, k:k + 16].t()
        top = torch.maximum(top, acc.abs())
    most = a.abs().max() * b.abs().max() if K and M else 0.0
    return acc, (top + most) * (17.0 * 2.0 ** -23 * -(-K // 16))


def rounded(v, e, dtype):
    """float64 v, known to e, rounded to dtype, and how far that rounding may be off."""
    mid, lo, hi = (t.to(dtype).double() for t in (v, v - e, v + e))
    return mid, torch.maximum((hi - mid).abs(), (mid - lo).abs())


def slack(d, other, chain):
    """``chain`` and what steps d [M, K] of the left operand can make of other [N, K]."""
    return chain + d @ other.abs().t()


def linear_fwd(x, w, b, res, name):
    z, e = product(x, w)
    if b is not None:
        z = z + b
        e = e + U * (z.abs() + e)
    (a, s), (ea, _) = act(name, z)
    # a slope of the activations is below 1.13 everywhere
    ey = 1.13 * e + ea
    y = a
    if res is not None:
        y = a + res
        ey = ey + U * (y.abs() + ey)
    return (y, z), (ey, e)


def linear_dz(g, z, name):
    if name == "none":
        return g, torch.zeros_like(g)
    (_, s), (_, es) = act(name, z)
    return g * s, g.abs() * es + 2.0 * U * (g * s).abs() + 2.0 ** -140


def linear_bwd(g, x, w, z, name, dtype, splits=64):
    """(dx, dw, db) and their bounds; ``splits``: at most so many parts of dw are added in fp32."""
    dz, e = linear_dz(g, z, name)
    d, step = (dz, torch.zeros_like(dz)) if name == "none" else rounded(dz, e, dtype)
    dx, edx = product(d, w.t())
    dw, edw = product(d.t(), x.t())
    edw = slack(step.t(), x.t(), 2.0 * edw) + splits * U * (d.abs().t() @ x.abs())
    # db: chains of at most T / 8 additions of a thread, then 8, 128 ranges' and their joins
    db = dz.sum(0)
    edb = e.sum(0) + (g.shape[0] / 8 + 300) * U * dz.abs().sum(0)
    return (dx, dw, db), (slack(step, w.t(), edx), edw, edb)


def gated_fwd(x, wg, wu, name):
    gate, eg = product(x, wg)
    up, eu = product(x, wu)
    (a, _), (ea, _) = act(name, gate)
    ea = ea + 1.13 * eg
    h = a * up
    eh = ea * up.abs() + a.abs() * eu + ea * eu + U * h.abs()
    return (h, gate, up), (eh, eg, eu)


def gated_bwd(g, x, wg, wu, gate, up, name, dtype, splits=64):
    (a, s), (ea, es) = act(name, gate)
    dup, edup = g * a, g.abs() * ea + 2.0 * U * (g * a).abs() + 2.0 ** -140
    dgate = g * s * up
    edgate = (g * up).abs() * es + 4.0 * U * dgate.abs() + 2.0 ** -140
    (dg, sg), (du, su) = rounded(dgate, edgate, dtype), rounded(dup, edup, dtype)
    # one chain over both products
    dx, edx = product(torch.cat((dg, du), 1), torch.cat((wg, wu), 0).t())
    edx = edx * (1.0 + 2.0 * 16.0 / max(g.shape[1], 1)) + sg @ wg.abs() + su @ wu.abs()
    out, err = [dx], [edx]
    for d, st in ((dg, sg), (du, su)):
        dw, edw = product(d.t(), x.t())
        out.append(dw)
        err.append(slack(st.t(), x.t(), 2.0 * edw) + splits * U * (d.abs().t() @ x.abs()))
    return out, err

