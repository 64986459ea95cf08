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
