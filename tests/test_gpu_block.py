"""A decoder block of this library's calls, forward and backward, as a program would
run them: norm, projection with bias, head norm with rotary positions of several
axes, (attention in plain torch), projection onto the residual stream, norm, gated
feed-forward block, projection onto the residual stream. Its outputs and every gradient
against automatic differentiation of the same block in 64 bits.

The bound: each of the block's 16-bit tensors is off by half a step, 2^-8 of a bf16 value at most, and on the way of any
gradient lie fewer than 24 of them (both ways through the block). Norms, activations and products pass a relative error on
with a factor of about one (rms to rms; a norm's backward takes a component out, the softmax's halves). 24 x 2^-8 is
0.09 of a tensor's size if all errors had one sign; they are taken together as rms.
"""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-6
BOUND = 24 * 2.0 ** -8


def _weights(E, Hq, Hk, D, F):
    m = lambda r, c, s: (synth.normal16((r, c), s, DEV, dtype=torch.float16).float() * c ** -0.5).to(BF16)
    return dict(wqkv=m((Hq + 2 * Hk) * D, E, 1), bqkv=synth.gamma_f32((Hq + 2 * Hk) * D, 2, DEV, mean=0.0, std=0.2),
                wo=m(E, Hq * D, 3), wg=m(F, E, 4), wu=m(F, E, 5), wd=m(E, F, 6), n1=synth.gamma_f32(E, 7, DEV), n2=synth.gamma_f32(E, 8, DEV),
                nq=synth.gamma_f32(D, 9, DEV), nk=synth.gamma_f32(D, 10, DEV))


def _attention(q, k, v):
    """Causal attention of grouped heads, [T, H, D]."""
    T, Hq, D = q.shape
    k, v = (t.repeat_interleave(Hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("thd,shd->hts", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return torch.einsum("hts,shd->thd", s.softmax(-1), v)


def _plain(x, w, f, axis, pos, Hq, Hk, D):
    """The block in 64 bits (x and w's tensors are leaves)."""
    T, E = x.shape

    def norm(t, g):
        return t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * g

    def turn(t):
        a = (pos[axis.long()].double().t() * f)[:, None]
        u, v = t.chunk(2, -1)
        return torch.cat((u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()), -1)

    qkv = norm(x, w["n1"]) @ w["wqkv"].t() + w["bqkv"]
    q, k, v = (t.reshape(T, -1, D) for t in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    o = _attention(turn(norm(q, w["nq"])), turn(norm(k, w["nk"])), v).reshape(T, Hq * D)
    x = x + o @ w["wo"].t()
    h = norm(x, w["n2"])
    return x + (torch.nn.functional.silu(h @ w["wg"].t()) * (h @ w["wu"].t())) @ w["wd"].t()


def _forward(x, w, f, axis, pos, Hq, Hk, D):
    T, E = x.shape
    F = w["wg"].shape[0]
    e = lambda *s: torch.empty(s, dtype=BF16, device=DEV)
    v = lambda *s: torch.empty(s, device=DEV)
    s = dict(x=x, a=e(T, E), r1=v(T), qkv=e(T, (Hq + 2 * Hk) * D), q=e(T, Hq, D), k=e(T, Hk, D), rq=v(T, Hq), rk=v(T, Hk), x1=e(T, E),
             h=e(T, E), r2=v(T), gate=e(T, F), up=e(T, F), u=e(T, F), y=e(T, E))
    rn.rmsnorm_fwd(x, w["n1"], s["a"], s["r1"], EPS)
    rn.linear_fwd(s["a"], w["wqkv"], w["bqkv"], None, s["qkv"])
    s["q0"], s["k0"] = s["qkv"][:, :Hq * D].view(T, Hq, D), s["qkv"][:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    s["v"] = s["qkv"][:, (Hq + Hk) * D:].view(T, Hk, D)
    rn.rmsnorm_rope_axes_fwd(s["q0"], s["k0"], w["nq"], w["nk"], f, axis, s["q"], s["k"], s["rq"], s["rk"], pos, eps=EPS)
    s["heads"] = [t.float().requires_grad_() for t in (s["q"], s["k"], s["v"])]
    with torch.enable_grad():
        s["att"] = _attention(*s["heads"])
    s["o"] = s["att"].detach().reshape(T, Hq * D).to(BF16)
    rn.linear_fwd(s["o"], w["wo"], None, x, s["x1"])
    rn.rmsnorm_fwd(s["x1"], w["n2"], s["h"], s["r2"], EPS)
    rn.linear_gated_fwd(s["h"], w["wg"], w["wu"], s["u"], s["gate"], s["up"])
    rn.linear_fwd(s["u"], w["wd"], None, s["x1"], s["y"])
    return s


def _backward(g, s, w, f, axis, pos, Hq, Hk, D):
    T, E = g.shape
    F, Q = w["wg"].shape[0], (Hq + 2 * Hk) * D
    e = lambda *sh: torch.empty(sh, dtype=BF16, device=DEV)
    d = {k: torch.empty_like(t) for k, t in w.items()}
    ws = torch.empty(max(rn.linear_bwd_workspace_bytes(T, E, F), rn.linear_gated_bwd_workspace_bytes(T, F, E), rn.workspace_bytes(T, E),
                         rn.linear_bwd_workspace_bytes(T, E, Hq * D), rn.linear_bwd_workspace_bytes(T, Q, E),
                         rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D)), dtype=torch.uint8, device=DEV)
    du, dh, dx1, do, dqkv, da, dx = e(T, F), e(T, E), e(T, E), e(T, Hq * D), e(T, Q), e(T, E), e(T, E)
    rn.linear_bwd(g, s["u"], w["wd"], None, du, d["wd"], None, ws)
    rn.linear_gated_bwd(du, s["h"], w["wg"], w["wu"], s["gate"], s["up"], dh, d["wg"], d["wu"], ws)
    rn.rmsnorm_residual_bwd(dh, s["x1"], w["n2"], s["r2"], g, dx1, d["n2"], ws)
    rn.linear_bwd(dx1, s["o"], w["wo"], None, do, d["wo"], None, ws)
    gq, gk, gv = (t.contiguous() for t in torch.autograd.grad(s["att"], s["heads"], do.float().view(T, Hq, D)))
    dq, dk = dqkv[:, :Hq * D].view(T, Hq, D), dqkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    dqkv[:, (Hq + Hk) * D:].view(T, Hk, D).copy_(gv)
    rn.rmsnorm_rope_axes_bwd(gq.to(BF16), gk.to(BF16), s["q0"], s["k0"], w["nq"], w["nk"], f, axis, s["rq"], s["rk"], dq, dk, d["nq"],
                             d["nk"], ws, pos)
    rn.linear_bwd(dqkv, s["a"], w["wqkv"], None, da, d["wqkv"], d["bqkv"], ws)
    rn.rmsnorm_residual_bwd(da, s["x"], w["n1"], s["r1"], dx1, dx, d["n1"], ws)
    return dx, d


@pytest.mark.parametrize("T,E,Hq,Hk,D,F", [(1, 256, 4, 2, 64, 520), (77, 512, 8, 2, 64, 1384), (300, 512, 4, 4, 128, 1032)])
def test_a_block_forward_and_backward(T, E, Hq, Hk, D, F):
    w = _weights(E, Hq, Hk, D, F)
    x, g = synth.normal16((T, E), 20, DEV), synth.normal16((T, E), 21, DEV)
    f = rn.rope_frequencies(D).to(DEV)
    axis = rn.rope_axes_map((D // 4, D // 8, D // 8), True).to(DEV)
    pos = torch.stack((torch.arange(T, device=DEV), torch.arange(T, device=DEV) // 16, torch.arange(T, device=DEV) % 16))
    s = _forward(x, w, f, axis, pos, Hq, Hk, D)
    dx, d = _backward(g, s, w, f, axis, pos, Hq, Hk, D)
    x64, w64 = x.double().requires_grad_(), {k: t.double().requires_grad_() for k, t in w.items()}
    y64 = _plain(x64, w64, f, axis, pos, Hq, Hk, D)
    y64.backward(g.double())
    for name, got, want in [("y", s["y"], y64.detach()), ("dx", dx, x64.grad)] + [("d" + k, d[k], w64[k].grad) for k in w]:
        size = float(want.norm())
        off = float((got.double() - want).norm())
        if T == 1 and name in ("dnq", "dnk"):  # one token attends to itself alone: the heads' gradients vanish
            assert float(got.abs().max()) <= 1e-5 and size <= 1e-12
            continue
        if T == 1 and name in ("dwqkv", "dbqkv"):  # of v alone
            continue
        assert off <= BOUND * size, (name, off / size)
    assert rn.rmsnorm_device_error() == 0


def test_a_row_of_the_block_does_not_depend_on_the_batch():
    """The rows of a longer batch through the calls without attention, bit for bit."""
    E, F = 512, 1384
    w = _weights(E, 4, 2, 64, F)

    def run(x):
        T = x.shape[0]
        e = lambda *s: torch.empty(s, dtype=BF16, device=DEV)
        a, u, y, r = e(T, E), e(T, F), e(T, E), torch.empty(T, device=DEV)
        rn.rmsnorm_fwd(x, w["n1"], a, r, EPS)
        rn.linear_gated_fwd(a, w["wg"], w["wu"], u)
        rn.linear_fwd(u, w["wd"], None, x, y)
        return y

    x = synth.normal16((3000, E), 30, DEV)
    whole = run(x)
    for n in (1, 7, 64, 130, 700):
        for first in (0, 1111, 3000 - n):
            assert torch.equal(run(x[first:first + n]).view(torch.int16), whole[first:first + n].view(torch.int16))
