"""Rotary positions of several axes, alone and fused with the head RMSNorm, on the
GPU: against the calls with one axis bit for bit, pair by pair, and against the
definitions in 64 bits (``tests/axes_ref.py``)."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests import axes_ref as ref
from tests.block_ref import assert_within, effective
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

EPS = 1e-6
F32_EPS = float(torch.tensor(EPS, dtype=torch.float32))
SCALE = 1.25  # exact in fp32
BF16, F16 = torch.bfloat16, torch.float16


def _bits(t):
    return t.contiguous().view(torch.int16)


def _heads(T, Hq, Hk, D, seed, dtype=BF16):
    """Views of one projection's output [T, (Hq + 2 Hk) D]."""
    t = synth.normal16((T, (Hq + 2 * Hk) * D), seed, DEV, dtype=dtype)
    return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None


def _pos(A, T, seed, dtype=torch.int64, layout="own"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    p = torch.randint(-(1 << 18), 1 << 20, (A, T), generator=g, device=DEV).to(dtype)
    if layout == "tokens":  # [T, axes] in memory
        return p.t().contiguous().t()
    if layout == "wide":    # every second token of longer rows
        wide = torch.full((A, 2 * T + 3), 7, dtype=dtype, device=DEV)
        wide[:, 1:2 * T:2] = p
        return wide[:, 1:2 * T:2]
    return p


def _sections(pairs, A):
    first = max(1, pairs - (A - 1) * (pairs // (A + 1)))
    rest = [max(1, pairs // (A + 1))] * (A - 1)
    return [pairs - sum(rest)] + rest if first else None


def _columns(axis, a, R, interleaved):
    """The values whose pairs are of axis a."""
    i = (axis.cpu() == a).nonzero().view(-1)
    return torch.cat((2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)).to(DEV)


def _buffers(q, k, g=None):
    e = lambda t: None if t is None else torch.empty_like(t.contiguous())
    r = lambda t: None if t is None else torch.empty(t.shape[:2], device=DEV)
    w = lambda t: None if t is None else torch.empty(t.shape[2], device=DEV)
    return e(q), e(k), r(q), r(k), w(q), w(k)


SHAPES = [(8, 8), (16, 12), (64, 64), (64, 32), (80, 32), (96, 24), (128, 128), (128, 78), (256, 64), (192, 36), (264, 264), (512, 512)]


@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,A,cycled,dtype,layout", [(1, 5, 1, 3, True, BF16, "own"), (67, 4, 2, 2, False, F16, "tokens"),
                                                           (33, 40, 0, 3, False, BF16, "wide"), (6005, 2, 1, 3, False, BF16, "tokens"),
                                                           (6007, 1, 0, 2, False, F16, "own")])
def test_every_pair_is_turned_by_its_axis(D, R, interleaved, T, Hq, Hk, A, cycled, dtype, layout):
    """Rotation, norm with rotation and (its weights' gradients) the norm's backward: the values of each axis's pairs are
    bit for bit those of the call with that axis's positions alone. One token a turn, and several (6005 tokens)."""
    if R // 2 < A + 1:
        A, cycled = 2, False
    q, k = _heads(T, Hq, Hk, D, D + R, dtype)
    gq, gk = _heads(T, Hq, Hk, D, D + R + 9, dtype)
    wq, wk = synth.gamma_f32(D, 1, DEV), synth.gamma_f32(D, 2, DEV) if Hk else None
    f = rn.rope_frequencies(R).to(DEV)
    axis = rn.rope_axes_map(_sections(R // 2, A), cycled).to(DEV)
    pos = _pos(A, T, R, torch.int32 if layout == "wide" else torch.int64, layout)
    ws = torch.full((max(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D) // 4, 4),), float("nan"), device=DEV)
    got, back, norm, grad = (_buffers(q, k) for _ in range(4))
    rn.rope_axes_fwd(q, k, f, axis, got[0], got[1], pos, SCALE, interleaved)
    rn.rope_axes_bwd(gq, gk, f, axis, back[0], back[1], pos, SCALE, interleaved)
    rn.rmsnorm_rope_axes_fwd(q, k, wq, wk, f, axis, *norm[:4], pos, SCALE, interleaved, EPS)
    rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, wq, wk, f, axis, norm[2], norm[3], *grad[:2], *grad[4:], ws, pos, SCALE, interleaved)
    rest = torch.arange(R, D, device=DEV)
    for a in range(A):
        p = pos[a].contiguous()
        got1, back1, norm1, grad1 = (_buffers(q, k) for _ in range(4))
        rn.rope_fwd(q, k, f, got1[0], got1[1], p, SCALE, interleaved)
        rn.rope_bwd(gq, gk, f, back1[0], back1[1], p, SCALE, interleaved)
        rn.rmsnorm_rope_fwd(q, k, wq, wk, f, *norm1[:4], p, SCALE, interleaved, EPS)
        rn.rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, f, norm1[2], norm1[3], *grad1[:2], *grad1[4:], ws, p, SCALE, interleaved)
        c = torch.cat((_columns(axis, a, R, interleaved), rest))
        for x, y in ((got, got1), (back, back1), (norm, norm1)):
            for i in (0, 1) if Hk else (0,):
                assert torch.equal(_bits(x[i][..., c]), _bits(y[i][..., c]))
        for i in (0, 1) if Hk else (0,):
            assert torch.equal(norm[2 + i], norm1[2 + i]) and torch.equal(grad[4 + i][c], grad1[4 + i][c])


@pytest.mark.parametrize("T,Hq,Hk,D,R,A,inter,cycled,dtype,zc", [
    (1, 5, 1, 128, 128, 3, False, True, BF16, False), (67, 32, 8, 128, 128, 3, False, False, F16, True),
    (300, 16, 2, 256, 64, 3, False, True, BF16, True), (500, 24, 24, 128, 128, 3, True, False, BF16, False),
    (6001, 1, 1, 64, 64, 2, True, False, F16, False), (6001, 4, 1, 128, 128, 3, False, True, BF16, False),
    (3001, 5, 0, 80, 72, 3, False, False, BF16, False), (33, 2, 2, 512, 510, 5, False, False, F16, False),
    (129, 3, 1, 96, 24, 2, True, True, BF16, True)])
def test_against_the_definition(T, Hq, Hk, D, R, A, inter, cycled, dtype, zc):
    q, k = _heads(T, Hq, Hk, D, 3, dtype)
    gq, gk = _heads(T, Hq, Hk, D, 4, dtype)
    mean = 0.0 if zc else 1.0
    wq, wk = synth.gamma_f32(D, 5, DEV, mean=mean, std=0.2), synth.gamma_f32(D, 6, DEV, mean=mean, std=0.2) if Hk else None
    f = rn.rope_frequencies(R, 500000.0).to(DEV)
    axis = rn.rope_axes_map(_sections(R // 2, A), cycled).to(DEV)
    pos = _pos(A, T, 8)
    got, norm, grad = (_buffers(q, k) for _ in range(3))
    rn.rope_axes_fwd(q, k, f, axis, got[0], got[1], pos, SCALE, inter)
    rn.rmsnorm_rope_axes_fwd(q, k, wq, wk, f, axis, *norm[:4], pos, SCALE, inter, EPS, zc)
    ws = torch.full((max(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D) // 4, 4),), float("nan"), device=DEV)
    rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, wq, wk, f, axis, norm[2], norm[3], *grad[:2], *grad[4:], ws, pos, SCALE, inter, zc)
    for i, (x, g, w) in enumerate(((q, gq, wq), (k, gk, wk))):
        if x is None:
            continue
        want, size = ref.turned(x.double(), pos, axis, f, SCALE, inter)
        assert_within("turned", got[i], want, ref.TURN * size, dtype)
        (want, rstd), (e, er) = ref.norm_turn_fwd(x.double(), effective(w, zc), F32_EPS, pos, axis, f, SCALE, inter)
        assert_within("norm", norm[i], want, e, dtype)
        assert_within("rstd", norm[2 + i], rstd, er)
        (want, rdw), (e, ew) = ref.norm_turn_bwd(g.double(), x.double(), effective(w, zc), norm[2 + i].double(), pos, axis, f,
                                                 SCALE, inter)
        assert_within("dx", grad[i], want, e, dtype)
        assert_within("dw", grad[4 + i], rdw, ew)


@pytest.mark.parametrize("T,Hq,Hk", [(50, 8, 2), (6001, 2, 1)])
def test_in_place(T, Hq, Hk):
    q, k = _heads(T, Hq, Hk, 128, 11)
    f, axis, pos = rn.rope_frequencies(128).to(DEV), rn.rope_axes_map((24, 20, 20), True).to(DEV), _pos(3, T, 12)
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    rn.rope_axes_fwd(q, k, f, axis, oq, ok, pos)
    rn.rope_axes_fwd(q, k, f, axis, q, k, pos)
    assert torch.equal(_bits(q), _bits(oq)) and torch.equal(_bits(k), _bits(ok))


def test_one_position_for_all_axes_or_tokens():
    """Strides of zero: all axes at one position (text), all tokens at one place."""
    T = 70
    q, k = _heads(T, 8, 2, 128, 13)
    f, axis = rn.rope_frequencies(128).to(DEV), rn.rope_axes_map((24, 20, 20)).to(DEV)
    p = _pos(1, T, 14)
    a, b, c = (_buffers(q, k)[:2] for _ in range(3))
    rn.rope_axes_fwd(q, k, f, axis, *a, p.expand(3, T))
    rn.rope_fwd(q, k, f, *b, p[0])
    assert torch.equal(_bits(a[0]), _bits(b[0])) and torch.equal(_bits(a[1]), _bits(b[1]))
    place = _pos(3, 1, 15)
    rn.rope_axes_fwd(q, k, f, axis, *a, place.expand(3, T))
    rn.rope_axes_fwd(q, k, f, axis, *c, place.expand(3, T).contiguous())
    assert torch.equal(_bits(a[0]), _bits(c[0])) and torch.equal(_bits(a[1]), _bits(c[1]))


@pytest.mark.parametrize("T,Hq,Hk", [(50, 8, 2), (6001, 2, 1)])
def test_an_axis_that_is_not_there_counts_as_the_last(T, Hq, Hk):
    q, k = _heads(T, Hq, Hk, 64, 16)
    f, pos = rn.rope_frequencies(64).to(DEV), _pos(2, T, 17)
    axis = torch.zeros(32, dtype=torch.uint8, device=DEV)
    axis[10:] = 1
    wild = axis.clone()
    wild[12:20], wild[20:] = 255, 2
    a, b = _buffers(q, k)[:2], _buffers(q, k)[:2]
    rn.rope_axes_fwd(q, k, f, axis, *a, pos)
    rn.rope_axes_fwd(q, k, f, wild, *b, pos)
    assert torch.equal(_bits(a[0]), _bits(b[0])) and torch.equal(_bits(a[1]), _bits(b[1]))


def test_no_tokens():
    q = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    f, axis, pos = rn.rope_frequencies(64).to(DEV), rn.rope_axes_map((16, 16)).to(DEV), _pos(2, 0, 1)
    w, dw, r = torch.ones(64, device=DEV), torch.ones(64, device=DEV), torch.empty((0, 4), device=DEV)
    rn.rope_axes_fwd(q, None, f, axis, q, None, pos)
    rn.rmsnorm_rope_axes_fwd(q, None, w, None, f, axis, q, None, r, None, pos)
    rn.rmsnorm_rope_axes_bwd(q, None, q, None, w, None, f, axis, r, None, q, None, dw, None, torch.empty(16, device=DEV), pos)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("T,Hq,Hk", [(40, 8, 2), (6001, 2, 1)])
def test_graph_and_another_stream(T, Hq, Hk):
    q, k = _heads(T, Hq, Hk, 128, 21)
    gq, gk = _heads(T, Hq, Hk, 128, 22)
    w = synth.gamma_f32(128, 23, DEV)
    f, axis, pos = rn.rope_frequencies(128).to(DEV), rn.rope_axes_map((24, 20, 20), True).to(DEV), _pos(3, T, 24)

    def buffers():
        return (*_buffers(q, k), torch.empty_like(q), torch.empty_like(k),
                torch.empty(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, 128), dtype=torch.uint8, device=DEV))

    def step(b):
        rn.rmsnorm_rope_axes_fwd(q, k, w, w, f, axis, *b[:4], pos)
        rn.rmsnorm_rope_axes_bwd(gq, gk, q, k, w, w, f, axis, b[2], b[3], b[6], b[7], b[4], b[5], b[8], pos)

    want, got, other = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step(other)
        with torch.cuda.graph(graph, stream=s):
            step(got)
    graph.replay()
    torch.cuda.synchronize()
    for b in (got, other):
        assert all(torch.equal(x, y) for x, y in zip(b[:8], want[:8]))
    pos.add_(5)
    graph.replay()
    step(want)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got[:8], want[:8]))


def test_the_binding_refuses_what_would_be_read_wrongly():
    q, k = _heads(8, 4, 2, 64, 31)
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    f, axis, pos = rn.rope_frequencies(64).to(DEV), rn.rope_axes_map((16, 8, 8)).to(DEV), _pos(3, 8, 32)
    for a, e in (((q, k, f, axis.long(), oq, ok, pos), TypeError), ((q, k, f, axis[:8], oq, ok, pos), TypeError),
                 ((q, k, f, axis.cpu(), oq, ok, pos), TypeError), ((q, k, f, axis, oq, ok, pos.float()), TypeError),
                 ((q, k, f, axis, oq, ok, pos.cpu()), TypeError), ((q, k, f, axis, oq, ok, pos[:, :4]), ValueError),
                 ((q, k, f, axis, oq, ok, pos[0]), ValueError), ((q, k, f, axis, oq, ok, pos[:0]), rn.RmsNormError),
                 ((q, k, f.float(), axis, oq, ok, pos), TypeError), ((q, k, f, axis, oq, None, pos), TypeError)):
        with pytest.raises(e):
            rn.rope_axes_fwd(*a)
