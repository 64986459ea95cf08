"""Gradients of the head norm with positions of several axes, dq and dk, over every
head width, rotated part, layout and kind of turn: against the definition in 64 bits, and, with
every axis at one position, against the call with one axis bit for bit."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests import axes_ref as ref
from tests.block_ref import assert_within, effective
from tests.gpu_common import DEV
from tests.test_gpu_rope_axes import BF16, EPS, F16, SCALE, SHAPES, _bits, _buffers, _heads, _pos, _sections

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,A,cycled,dtype,layout,zc", [
    (1, 5, 1, 3, True, BF16, "own", True), (67, 4, 2, 2, False, F16, "tokens", False), (33, 40, 0, 3, False, BF16, "wide", False),
    (6005, 2, 1, 3, False, BF16, "tokens", False), (6007, 1, 0, 2, False, F16, "own", True)])
def test_dq_and_dk(D, R, interleaved, T, Hq, Hk, A, cycled, dtype, layout, zc):
    if R // 2 < A + 1:
        A, cycled = 2, False
    q, k = _heads(T, Hq, Hk, D, D + R, dtype)
    gq, gk = _heads(T, Hq, Hk, D, D + R + 9, dtype)
    mean = 0.0 if zc else 1.0
    wq, wk = synth.gamma_f32(D, 1, DEV, mean=mean, std=0.2), synth.gamma_f32(D, 2, DEV, mean=mean, std=0.2) if Hk else None
    f = rn.rope_frequencies(R).to(DEV)
    axis = rn.rope_axes_map(_sections(R // 2, A), cycled).to(DEV)
    pos = _pos(A, T, R, torch.int32 if layout == "wide" else torch.int64, layout)
    ws = torch.full((max(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D) // 4, 4),), float("nan"), device=DEV)
    norm = _buffers(q, k)
    rn.rmsnorm_rope_axes_fwd(q, k, wq, wk, f, axis, *norm[:4], pos, SCALE, interleaved, EPS, zc)

    def poisoned():
        b = _buffers(q, k)
        for t in b:
            if t is not None:
                t.fill_(float("nan"))
        return b

    grad = poisoned()
    rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, wq, wk, f, axis, norm[2], norm[3], *grad[:2], *grad[4:], ws, pos, SCALE, interleaved, zc)
    for i, (x, g, w) in enumerate(((q, gq, wq), (k, gk, wk))):
        if x is not None:
            (want, _), (e, _) = ref.norm_turn_bwd(g.double(), x.double(), effective(w, zc), norm[2 + i].double(), pos, axis, f, SCALE,
                                                  interleaved)
            assert_within("dq" if i == 0 else "dk", grad[i], want, e, dtype)
    # one position for all axes: the call with one axis
    p = pos[0].contiguous()
    several, one = poisoned(), poisoned()
    rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, wq, wk, f, axis, norm[2], norm[3], *several[:2], *several[4:], ws, p[None].expand(A, T),
                             SCALE, interleaved, zc)
    rn.rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, f, norm[2], norm[3], *one[:2], *one[4:], ws, p, SCALE, interleaved, zc)
    for i in (0, 1) if Hk else (0,):
        assert torch.equal(_bits(several[i]), _bits(one[i])) and torch.equal(several[4 + i], one[4 + i])


@pytest.mark.parametrize("D,R", [(64, 64), (80, 72), (128, 78), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk", [(50, 8, 2), (6001, 2, 1)])
def test_in_place_and_beside_other_columns(D, R, interleaved, T, Hq, Hk):
    """Gradients written over those of the outputs, and every output as part of one projection's buffer whose
    other columns stay as they were: the bits of outputs of their own."""
    q, k = _heads(T, Hq, Hk, D, 41)
    gq, gk = _heads(T, Hq, Hk, D, 42)
    w = synth.gamma_f32(D, 43, DEV)
    f, axis, pos = rn.rope_frequencies(R).to(DEV), rn.rope_axes_map(_sections(R // 2, 3)).to(DEV), _pos(3, T, 44)
    ws = torch.full((max(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D) // 4, 4),), float("nan"), device=DEV)
    rq, rk, dw = torch.empty((T, Hq), device=DEV), torch.empty((T, Hk), device=DEV), [torch.empty(D, device=DEV) for _ in range(2)]
    calls = (lambda a, b: rn.rope_axes_fwd(q, k, f, axis, a, b, pos, SCALE, interleaved),
             lambda a, b: rn.rope_axes_bwd(gq, gk, f, axis, a, b, pos, SCALE, interleaved),
             lambda a, b: rn.rmsnorm_rope_axes_fwd(q, k, w, w, f, axis, a, b, rq, rk, pos, SCALE, interleaved, EPS),
             lambda a, b: rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, w, w, f, axis, rq, rk, a, b, *dw, ws, pos, SCALE, interleaved))
    for call in calls:
        own = _buffers(q, k)[:2]
        call(*own)
        base = torch.full((T, (Hq + 2 * Hk) * D + 16), 3.0, dtype=BF16, device=DEV)
        a, b = base[:, 8:8 + Hq * D].view(T, Hq, D), base[:, 8 + (Hq + Hk) * D:8 + (Hq + 2 * Hk) * D].view(T, Hk, D)
        call(a, b)
        assert torch.equal(_bits(a), _bits(own[0])) and torch.equal(_bits(b), _bits(own[1]))
        rest = torch.cat((base[:, :8], base[:, 8 + Hq * D:8 + (Hq + Hk) * D], base[:, -8:]), 1)
        assert bool((rest == 3.0).all())
    want, turned = _buffers(q, k)[:2], _buffers(q, k)[:2]
    calls[3](*want)
    sums = [t.clone() for t in dw]
    calls[1](*turned)
    pq, pk = gq.clone(), gk.clone()
    rn.rope_axes_bwd(pq, pk, f, axis, pq, pk, pos, SCALE, interleaved)
    assert torch.equal(_bits(pq), _bits(turned[0])) and torch.equal(_bits(pk), _bits(turned[1]))
    calls[3](gq, gk)  # over the gradients themselves
    assert torch.equal(_bits(gq), _bits(want[0])) and torch.equal(_bits(gk), _bits(want[1]))
    assert torch.equal(dw[0], sums[0]) and torch.equal(dw[1], sums[1])
