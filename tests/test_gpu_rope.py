"""Rotary positions, alone and fused with the head RMSNorm of q and k, on the GPU
against their definitions in 64 bits (``tests/block_ref.py``)."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests import block_ref as ref
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

EPS = 1e-6
F32_EPS = float(torch.tensor(EPS, dtype=torch.float32))
SCALE = 1.25  # exact in fp32
BF16, F16 = torch.bfloat16, torch.float16


def _bits(t):
    return t.contiguous().view(torch.int16)


def _heads(T, Hq, Hk, D, seed, dtype=BF16, layout="own"):
    """q and k: tensors of their own, views of one projection's output [T, (Hq + 2 Hk) D], or with the heads
    outermost ([H, T, D] in memory)."""
    if layout == "qkv":
        t = synth.normal16((T, (Hq + 2 * Hk) * D), seed, DEV, dtype=dtype)
        return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None
    if layout == "heads":
        q = synth.normal16((Hq, T, D), seed, DEV, dtype=dtype).transpose(0, 1)
        return q, synth.normal16((Hk, T, D), seed + 1, DEV, dtype=dtype).transpose(0, 1) if Hk else None
    return synth.normal16((T, Hq, D), seed, DEV, dtype=dtype), \
        synth.normal16((T, Hk, D), seed + 1, DEV, dtype=dtype) if Hk else None


def _like(t, fill=3.0):
    """An output of t's shape and strides inside a buffer of ``fill``."""
    if t is None:
        return None, None
    n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 1
    base = torch.full((n + 64,), fill, dtype=t.dtype, device=DEV)
    return base, base.as_strided(t.shape, t.stride())


def _beside(base, out):
    """What of ``base`` lies outside ``out``."""
    keep = torch.ones(base.numel(), dtype=torch.bool, device=DEV)
    keep.as_strided(out.shape, out.stride()).fill_(False)
    return base[keep]


def _pos(T, seed, span=1 << 20, dtype=torch.int64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-span // 4, span, (T,), generator=g, device=DEV).to(dtype)


def _freq(R, theta=10000.0, **kw):
    return rn.rope_frequencies(R, theta, **kw).to(DEV)


# (D, R): whole heads and parts, pairs that fill 16-byte vectors and pairs that do not
SHAPES = [(8, 2), (8, 8), (16, 16), (24, 24), (64, 64), (64, 32), (72, 72), (80, 32), (96, 24), (96, 96), (128, 128),
          (128, 64), (128, 78), (128, 126), (128, 2), (192, 192), (192, 64), (256, 64), (256, 256), (256, 250),
          (264, 264), (320, 320), (512, 512), (512, 64), (512, 510), (512, 2),
          (512, 34), (496, 490), (40, 36), (160, 160), (128, 36), (128, 44)]


@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,dtype,layout", [(1, 5, 1, BF16, "own"), (67, 4, 2, F16, "qkv"),
                                                  (33, 3, 0, BF16, "heads")])
def test_rope(D, R, interleaved, T, Hq, Hk, dtype, layout):
    q, k = _heads(T, Hq, Hk, D, D + R, dtype, layout)
    pos, f = _pos(T, R, dtype=torch.int32 if T == 67 else torch.int64), _freq(R)
    for back in (False, True):
        bq, oq = _like(q)
        bk, ok = _like(k)
        (rn.rope_bwd if back else rn.rope_fwd)(q, k, f, oq, ok, pos, SCALE, interleaved)
        for name, x, base, o in (("q", q, bq, oq), ("k", k, bk, ok)):
            if x is None:
                continue
            want, size = ref.turned(x.double(), pos, f, SCALE, interleaved, back)
            ref.assert_within(name, o, want, ref.TURN * size, dtype)
            assert torch.equal(_bits(o[..., R:]), _bits(x[..., R:]))
            assert bool((_beside(base, o) == 3.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (96, 24), (256, 250)])
def test_rope_in_place(D, R, interleaved):
    q, k = _heads(130, 4, 2, D, 3, BF16, "qkv")
    pos, f = _pos(130, 4), _freq(R)
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    rn.rope_fwd(q, k, f, oq, ok, pos, SCALE, interleaved)
    rn.rope_fwd(q, k, f, q, k, pos, SCALE, interleaved)
    assert torch.equal(_bits(q), _bits(oq)) and torch.equal(_bits(k), _bits(ok))


def test_far_positions():
    """Positions up to 2^31 and of either sign turn by their angle modulo one turn: the 64-bit product is exact, so
    frequencies of a whole fraction of a turn give exact places on the circle."""
    turn = 6.283185307179586476925
    f = torch.tensor([turn / 4, turn / 8, turn / 2 ** 20], dtype=torch.float64, device=DEV)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 2 ** 40 + 3], device=DEV)
    x = torch.zeros((7, 1, 8), dtype=F16, device=DEV)
    x[..., 0:3] = 1.0  # pairs (1, 0)
    o, _ = _like(x)[1], None
    rn.rope_fwd(x, None, f, o, None, pos)
    for j, n in enumerate((4, 8, 2 ** 20)):
        a = torch.remainder(pos, n).double() * (turn / n)
        # the frequency's fp64 rounding, |a| 2^-52, reaches 2^-10 at 2^40: below half a step of fp16 at 1 for n = 4, 8
        err = ref.TURN + (pos.double().abs() * (turn / n)) * 2.0 ** -51
        ref.assert_within(f"cos {n}", o[:, 0, j], a.cos(), err, F16)
        ref.assert_within(f"sin {n}", o[:, 0, 3 + j], a.sin(), err, F16)


def test_positions_default_and_types():
    q, k = _heads(300, 4, 1, 64, 9)
    f = _freq(64)
    outs = []
    for pos in (None, torch.arange(300, device=DEV), torch.arange(300, device=DEV, dtype=torch.int32)):
        oq, ok = torch.empty_like(q), torch.empty_like(k)
        rn.rope_fwd(q, k, f, oq, ok, pos)
        outs.append((oq, ok))
    for oq, ok in outs[1:]:
        assert torch.equal(_bits(oq), _bits(outs[0][0])) and torch.equal(_bits(ok), _bits(outs[0][1]))


def test_backward_undoes_forward():
    q, _ = _heads(64, 8, 0, 128, 13, F16)
    f, pos = _freq(128, 500000.0, scaling="ramp_turns", factor=8.0, low=4.0, high=32.0, length=8192.0), _pos(64, 14)
    o = torch.empty_like(q)
    rn.rope_fwd(q, None, f, o, None, pos)
    back = torch.empty_like(q)
    rn.rope_bwd(o, None, f, back, None, pos)
    # two roundings to fp16 of values of at most |u| + |v|, the first turned again
    size = ref.turned(q.double(), pos, f, 1.0, False)[1]
    ref.assert_within("q", back, q.double(), size * (2 * ref.TURN + 2.0 ** -10), F16)


def test_nan_and_infinity_stay_in_their_pair():
    q, _ = _heads(4, 2, 0, 128, 17)
    q[1, 0, 5] = float("nan")
    q[2, 1, 100] = float("inf")   # outside the turned part
    for inter in (False, True):
        o = torch.empty_like(q)
        rn.rope_fwd(q, None, _freq(64), o, None, None, 1.0, inter)
        bad = ~o.isfinite()
        want = torch.zeros_like(bad)
        want[1, 0, [4, 5] if inter else [5, 37]] = True
        want[2, 1, 100] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("Hq,Hk", [(1, 0), (1, 1), (7, 3), (40, 1), (2, 33), (128, 8)])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (64, 64, True), (96, 24, False), (256, 64, False), (16, 16, False)])
def test_any_number_of_heads(Hq, Hk, D, R, inter):
    """Turns of warps that are not full, of q, of k and of both; more tokens than a batch of positions."""
    for T in (1, 45, 400):
        _check_norm(T, Hq, Hk, D, R, inter, BF16, "qkv", False, seed=T)


def test_more_than_two_to_the_31_values():
    """The last tokens of tensors of more than 2^31 values, against the same tokens on their own."""
    T, H, D, R = (1 << 31) // (32 * 512) + 7, 32, 512, 512
    tq, _ = _heads(3, H, 0, D, 93)
    tg, _ = _heads(3, H, 0, D, 94)
    q = torch.zeros((T, H, D), dtype=BF16, device=DEV)
    g = torch.zeros((T, H, D), dtype=BF16, device=DEV)
    q[-3:], g[-3:] = tq, tg
    w, _ = _weights(D, 0, 95, False)
    f = _freq(R)
    pos = torch.arange(T, device=DEV)
    o, d = torch.empty_like(q), torch.empty_like(q)
    rstd, dw = torch.empty((T, H), device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(rn.rmsnorm_rope_bwd_workspace_bytes(T, H, 0, D), dtype=torch.uint8, device=DEV)
    rn.rmsnorm_rope_fwd(q, None, w, None, f, o, None, rstd, None, pos, SCALE, False, EPS)
    (_, to, tr), _ = _norm_fwd(tq, None, w, None, f, pos[-3:].clone())
    assert torch.equal(_bits(o[-3:]), _bits(to)) and torch.equal(rstd[-3:], tr)
    rn.rmsnorm_rope_bwd(g, None, q, None, w, None, f, rstd, None, d, None, dw, None, ws, pos, SCALE, False)
    (_, td, tdw), _ = _norm_bwd(tg, None, tq, None, w, None, f, tr, None, pos[-3:].clone())
    assert torch.equal(_bits(d[-3:]), _bits(td))
    torch.testing.assert_close(dw, tdw, rtol=1e-4, atol=1e-4)  # 96 rows in another order, the others zero
    rn.rope_fwd(q, None, f, o, None, pos, SCALE)
    to2 = torch.empty_like(tq)
    rn.rope_fwd(tq, None, f, to2, None, pos[-3:].clone(), SCALE)
    assert torch.equal(_bits(o[-3:]), _bits(to2))


def test_two_streams_at_once():
    """Two backwards that overlap, each with a workspace of its own."""
    T, D = 3000, 128
    runs = []
    for seed in (101, 102):
        q, k = _heads(T, 8, 2, D, seed)
        g, h = _heads(T, 8, 2, D, seed + 10)
        wq, wk = _weights(D, 2, seed, False)
        (_, _, r), (_, _, rk) = _norm_fwd(q, k, wq, wk, _freq(D), None)
        runs.append((g, h, q, k, wq, wk, _freq(D), r, rk, None))
    alone = [_norm_bwd(*a) for a in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        got = []
        for st, a in zip(streams, runs):
            with torch.cuda.stream(st):
                got.append(_norm_bwd(*a))
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            for i in (0, 1):
                assert torch.equal(_bits(x[i][1]), _bits(y[i][1])) and torch.equal(x[i][2], y[i][2])


def test_the_binding_refuses_what_would_be_read_wrongly():
    q, k = _heads(8, 4, 2, 64, 111)
    f = _freq(64)
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    p = torch.arange(8, device=DEV)
    for a, e in (((q.float(), k, f, oq, ok, p), TypeError), ((q, k.half(), f, oq, ok, p), TypeError),
                 ((q, k.cpu(), f, oq, ok, p), TypeError), ((q, k, f.float(), oq, ok, p), TypeError),
                 ((q, k, f.cpu(), oq, ok, p), TypeError), ((q, k, f, oq, ok, p.float()), TypeError),
                 ((q, k, f, oq, ok, p[:4]), TypeError), ((q, k, f, oq, None, p), TypeError),
                 ((q, k, f, oq[:, :2], ok, p), ValueError), ((q, k[:4], f, oq, ok, p), ValueError),
                 ((q.transpose(1, 2), None, f, oq, None, p), ValueError), ((q[0], None, f, oq, None, p), TypeError),
                 ((q, None, f[None], oq, None, p), TypeError), ((q, k, _freq(66), oq, ok, p), rn.RmsNormError)):
        with pytest.raises(e):
            rn.rope_fwd(*a)
    wq, wk = _weights(64, 2, 5, False)
    rq, rk = torch.empty((8, 4), device=DEV), torch.empty((8, 2), device=DEV)
    for bad in (dict(wk=None), dict(wq=wq.half()), dict(rk=rk[:, :1]), dict(rq=rq.t())):
        a = {**dict(wq=wq, wk=wk, rq=rq, rk=rk), **bad}
        with pytest.raises(TypeError):
            rn.rmsnorm_rope_fwd(q, k, a["wq"], a["wk"], f, oq, ok, a["rq"], a["rk"], p)


def test_shared_heads_and_broadcast_inputs():
    """An input of stride 0 over its heads is read once for each of them."""
    x = synth.normal16((50, 1, 64), 5, DEV)
    o, w = torch.empty((50, 6, 64), dtype=BF16, device=DEV), torch.empty((50, 6, 64), dtype=BF16, device=DEV)
    rn.rope_fwd(x.expand(50, 6, 64), None, _freq(64), o, None)
    rn.rope_fwd(x.expand(50, 6, 64).contiguous(), None, _freq(64), w, None)
    assert torch.equal(_bits(o), _bits(w))


# --------------------------------------------------------------------------
# fused with the head norm
# --------------------------------------------------------------------------
def _weights(D, Hk, seed, zc):
    w = [synth.gamma_f32(D, seed + i, DEV, mean=0.0 if zc else 1.0, std=0.2) for i in (0, 1)]
    return w[0], w[1] if Hk else None


def _norm_fwd(q, k, wq, wk, f, pos, inter=False, zc=False, scale=SCALE):
    T, Hq = q.shape[:2]
    bq, oq = _like(q)
    bk, ok = _like(k)
    rq = torch.empty((T, Hq), device=DEV)
    rk = torch.empty((T, k.shape[1]), device=DEV) if k is not None else None
    rn.rmsnorm_rope_fwd(q, k, wq, wk, f, oq, ok, rq, rk, pos, scale, inter, EPS, zc)
    return (bq, oq, rq), (bk, ok, rk)


def _norm_bwd(gq, gk, q, k, wq, wk, f, rq, rk, pos, inter=False, zc=False, scale=SCALE):
    T, Hq, D = q.shape
    Hk = 0 if k is None else k.shape[1]
    bq, dq = _like(gq)
    bk, dk = _like(gk)
    dwq = torch.full((D,), 5.0, device=DEV)
    dwk = torch.full((D,), 5.0, device=DEV) if Hk else None
    ws = torch.full((max(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D) // 4, 4),), float("nan"), device=DEV)
    rn.rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, f, rq, rk, dq, dk, dwq, dwk, ws, pos, scale, inter, zc)
    return (bq, dq, dwq), (bk, dk, dwk)


def _check_norm(T, Hq, Hk, D, R, inter, dtype, layout, zc, seed=0):
    q, k = _heads(T, Hq, Hk, D, D + R + seed, dtype, layout)
    gq, gk = _heads(T, Hq, Hk, D, D + R + seed + 50, dtype, "own" if layout == "heads" else layout)
    wq, wk = _weights(D, Hk, seed + 7, zc)
    pos, f = _pos(T, R + seed), _freq(R)
    outs = _norm_fwd(q, k, wq, wk, f, pos, inter, zc)
    rq, rk = outs[0][2], outs[1][2]
    for name, x, w, (base, o, r) in (("q", q, wq, outs[0]), ("k", k, wk, outs[1])):
        if x is None:
            continue
        (want, rstd), (e, er) = ref.norm_turn_fwd(x.double(), ref.effective(w, zc), F32_EPS, pos, f, SCALE, inter)
        ref.assert_within(f"rstd {name}", r, rstd, er)
        ref.assert_within(name, o, want, e, dtype)
        assert bool((_beside(base, o) == 3.0).all())
    outs = _norm_bwd(gq, gk, q, k, wq, wk, f, rq, rk, pos, inter, zc)
    for name, g, x, w, r, (base, d, dw) in (("q", gq, q, wq, rq, outs[0]), ("k", gk, k, wk, rk, outs[1])):
        if x is None:
            continue
        (want, rdw), (e, ew) = ref.norm_turn_bwd(g.double(), x.double(), ref.effective(w, zc), r.double(), pos, f,
                                                 SCALE, inter)
        ref.assert_within(f"d{name}", d, want, e, dtype)
        ref.assert_within(f"dw{name}", dw, rdw, ew)
        assert bool((_beside(base, d) == 3.0).all())


@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,dtype,layout,zc", [(1, 5, 1, BF16, "own", False), (67, 4, 2, F16, "qkv", True),
                                                     (33, 3, 0, BF16, "heads", False)])
def test_norm_and_rope(D, R, interleaved, T, Hq, Hk, dtype, layout, zc):
    _check_norm(T, Hq, Hk, D, R, interleaved, dtype, layout, zc)


@pytest.mark.parametrize("T,Hq,Hk,D,R", [(4093, 16, 2, 256, 64), (3001, 32, 8, 128, 128), (20011, 2, 1, 64, 64),
                                         (1000, 56, 8, 96, 24), (700, 7, 7, 512, 512)])
@pytest.mark.parametrize("dtype,interleaved", [(BF16, False), (F16, True)])
def test_norm_and_rope_many_tokens(T, Hq, Hk, D, R, dtype, interleaved):
    _check_norm(T, Hq, Hk, D, R, interleaved, dtype, "qkv", dtype == F16, seed=T)


@pytest.mark.parametrize("Hq,Hk", [(1, 0), (1, 1), (2, 1), (4, 1), (5, 0), (7, 1), (3, 2), (14, 2)])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 20, True), (8, 8, True),
                                       (24, 24, False), (80, 32, False), (96, 24, False), (128, 78, False),
                                       (256, 64, False), (256, 256, True), (192, 36, False), (264, 264, False)])
def test_few_heads_and_many_tokens(Hq, Hk, D, R, inter):
    """Turns of several tokens, the last of which are not there; heads of their own and of a wider projection."""
    T = 6001 + 2 * Hq
    _check_norm(T, Hq, Hk, D, R, inter, F16 if Hq == 2 else BF16, "heads" if Hq == 3 else "own" if Hq == 4 else "qkv",
                False, seed=Hq)
    q, k = _heads(T, Hq, Hk, D, 3, BF16, "qkv" if Hq == 4 else "own")
    pos, f = _pos(T, 5), _freq(R)
    for back in (False, True):
        bq, oq = _like(q)
        bk, ok = _like(k)
        (rn.rope_bwd if back else rn.rope_fwd)(q, k, f, oq, ok, pos, SCALE, inter)
        for name, x, base, o in (("q", q, bq, oq), ("k", k, bk, ok)):
            if x is not None:
                want, size = ref.turned(x.double(), pos, f, SCALE, inter, back)
                ref.assert_within(name, o, want, ref.TURN * size, BF16)
                assert torch.equal(_bits(o[..., R:]), _bits(x[..., R:]))
                assert bool((_beside(base, o) == 3.0).all())


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (256, 64, False), (128, 128, True), (96, 24, False)])
def test_norm_and_rope_rows_are_their_own(D, R, inter):
    """A token's bits do not depend on the batch, its place, the strides, the other heads or bad values beside it."""
    q0, k0 = _heads(1, 4, 2, D, 1)
    g0, h0 = _heads(1, 4, 2, D, 3)
    wq, wk = _weights(D, 2, 5, False)
    f, p0 = _freq(R), _pos(1, 6)
    (_, o1, r1), (_, ok1, rk1) = _norm_fwd(q0, k0, wq, wk, f, p0, inter)
    (_, d1, _), (_, dk1, _) = _norm_bwd(g0, h0, q0, k0, wq, wk, f, r1, rk1, p0, inter)
    for T, at in ((2, 1), (33, 17), (700, 699), (5000, 2501)):
        for layout in ("own", "qkv", "heads"):
            q, k = _heads(T, 4, 2, D, T, BF16, layout)
            g, h = _heads(T, 4, 2, D, T + 1, BF16, layout)
            pos = _pos(T, T)
            q[at], k[at], g[at], h[at], pos[at] = q0[0], k0[0], g0[0], h0[0], p0[0]
            if T > 2:
                q[at - 1, 0] = float("nan")
                g[at - 1, 1, 3] = float("inf")
            (_, o, r), (_, ok, rk) = _norm_fwd(q, k, wq, wk, f, pos, inter)
            (_, d, _), (_, dk, _) = _norm_bwd(g, h, q, k, wq, wk, f, r, rk, pos, inter)
            for a, b in ((o, o1), (ok, ok1), (d, d1), (dk, dk1)):
                assert torch.equal(_bits(a[at]), _bits(b[0]))
            assert torch.equal(r[at], r1[0]) and torch.equal(rk[at], rk1[0])


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 64, True), (96, 24, False)])
def test_norm_and_rope_in_place(D, R, inter):
    T = 200
    q, k = _heads(T, 4, 2, D, 3, BF16, "qkv")
    g, h = _heads(T, 4, 2, D, 5, BF16, "qkv")
    wq, wk = _weights(D, 2, 5, False)
    f, pos = _freq(R), _pos(T, 4)
    (_, o, r), (_, ok, rk) = _norm_fwd(q, k, wq, wk, f, pos, inter)
    (_, d, dw), (_, dk, dwk) = _norm_bwd(g, h, q, k, wq, wk, f, r, rk, pos, inter)
    ws = torch.empty(rn.rmsnorm_rope_bwd_workspace_bytes(T, 4, 2, D), dtype=torch.uint8, device=DEV)
    dw2, dwk2 = torch.empty_like(dw), torch.empty_like(dwk)
    rn.rmsnorm_rope_bwd(g, h, q, k, wq, wk, f, r, rk, g, h, dw2, dwk2, ws, pos, SCALE, inter, False)
    assert torch.equal(_bits(g), _bits(d)) and torch.equal(_bits(h), _bits(dk))
    assert torch.equal(dw, dw2) and torch.equal(dwk, dwk2)
    r2, rk2 = torch.empty_like(r), torch.empty_like(rk)
    rn.rmsnorm_rope_fwd(q, k, wq, wk, f, q, k, r2, rk2, pos, SCALE, inter, EPS, False)
    assert torch.equal(_bits(q), _bits(o)) and torch.equal(_bits(k), _bits(ok)) and torch.equal(r, r2)


def test_fused_call_agrees_with_the_norm_and_the_rotation():
    """The fused forward is rmsnorm_fwd then rope_fwd but for the 16-bit rounding between them, and their rstd is
    the same sum in another order."""
    T, H, D = 500, 4, 128
    q, _ = _heads(T, H, 0, D, 61)
    w, _ = _weights(D, 0, 62, True)
    f, pos = _freq(D), _pos(T, 63)
    (_, o, r), _ = _norm_fwd(q, None, w, None, f, pos, zc=True, scale=1.0)
    y, rstd = torch.empty_like(q), torch.empty(T * H, device=DEV)
    rn.rmsnorm_fwd(q.view(-1, D), w, y.view(-1, D), rstd, EPS, True)
    two = torch.empty_like(q)
    rn.rope_fwd(y, None, f, two, None, pos)
    ref.assert_within("rstd", r.view(-1), rstd.double(), rstd.double() * (2 * (ref.K + 3) * ref.U + 2 * ref.RSQRT))
    _, size = ref.turned(y.double(), pos, f, 1.0, False)
    # y's rounding (2^-9 of each value) turned, both calls' fp32 errors, and one rounding of each output
    ref.assert_within("q", o, two.double(), size * (2.0 ** -8 + 2.0 ** -17) + two.double().abs() * 2.0 ** -8, BF16)


def test_norm_and_rope_weight_gradients_repeat():
    T, D = 3000, 128
    q, k = _heads(T, 8, 2, D, 71)
    g, h = _heads(T, 8, 2, D, 72)
    wq, wk = _weights(D, 2, 73, False)
    f = _freq(D)
    (_, _, r), (_, _, rk) = _norm_fwd(q, k, wq, wk, f, None)
    first = _norm_bwd(g, h, q, k, wq, wk, f, r, rk, None)
    for _ in range(3):
        again = _norm_bwd(g, h, q, k, wq, wk, f, r, rk, None)
        assert torch.equal(first[0][2], again[0][2]) and torch.equal(first[1][2], again[1][2])


def test_the_entry_points_called_with_their_own_arguments():
    """The C entry points, which the binding calls with an array, argument by argument: the same bits."""
    lib, st = rn.load(), torch.cuda.current_stream().cuda_stream
    T, Hq, Hk, D = 37, 4, 2, 64
    q, k = _heads(T, Hq, Hk, D, 121, F16, "qkv")
    g, h = _heads(T, Hq, Hk, D, 122, F16)
    wq, wk = _weights(D, Hk, 123, True)
    f, pos = _freq(32), _pos(T, 124)
    W = (Hq + 2 * Hk) * D

    def p(t):
        return t.data_ptr()

    (_, o, r), (_, ok, rk) = _norm_fwd(q, k, wq, wk, f, pos, True, True)
    (_, d, dw), (_, dk, dwk) = _norm_bwd(g, h, q, k, wq, wk, f, r, rk, pos, True, True)
    o2, ok2, d2, dk2 = (torch.empty((T, n, D), dtype=F16, device=DEV) for n in (Hq, Hk, Hq, Hk))
    r2, rk2 = torch.empty_like(r), torch.empty_like(rk)
    dw2, dwk2 = torch.empty_like(dw), torch.empty_like(dwk)
    own = ((Hq * D, D), (Hk * D, D))
    assert lib.rmsnorm_rope_fwd(p(q), W, D, p(k), W, D, p(wq), p(wk), p(f), p(pos), 1, p(o2), *own[0], p(ok2), *own[1],
                                p(r2), p(rk2), T, Hq, Hk, D, 32, SCALE, 1, EPS, 1, 1, st) == 0
    ws = torch.empty(rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D), dtype=torch.uint8, device=DEV)
    assert lib.rmsnorm_rope_bwd(p(g), *own[0], p(h), *own[1], p(q), W, D, p(k), W, D, p(wq), p(wk), p(f), p(pos), 1,
                                p(r2), p(rk2), p(d2), *own[0], p(dk2), *own[1], p(dw2), p(dwk2), p(ws), ws.numel(), T,
                                Hq, Hk, D, 32, SCALE, 1, 1, 1, st) == 0
    for a, b in ((o, o2), (ok, ok2), (d, d2), (dk, dk2)):
        assert torch.equal(_bits(a), _bits(b))
    for a, b in ((r, r2), (rk, rk2), (dw, dw2), (dwk, dwk2)):
        assert torch.equal(a, b)
    for fn in ("rope_fwd", "rope_bwd"):
        getattr(rn, fn)(q, k, f, o2, ok2, pos, SCALE, True)
        assert getattr(lib, fn)(p(q), W, D, p(k), W, D, p(f), p(pos), 1, p(d2), *own[0], p(dk2), *own[1], T, Hq, Hk, D, 32,
                                SCALE, 1, 1, st) == 0
        assert torch.equal(_bits(o2), _bits(d2)) and torch.equal(_bits(ok2), _bits(dk2))


def test_no_tokens():
    q, k = _heads(0, 4, 2, 64, 1)
    f = _freq(64)
    rn.rope_fwd(q, k, f, torch.empty_like(q), torch.empty_like(k))
    wq, wk = _weights(64, 2, 5, False)
    (_, _, r), (_, _, rk) = _norm_fwd(q, k, wq, wk, f, None)
    (_, _, dwq), (_, _, dwk) = _norm_bwd(q, k, q, k, wq, wk, f, r, rk, None)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())


@pytest.mark.parametrize("T", [3, 2000])
def test_a_block_of_them_captured_and_replayed(T):
    """LayerNorm, the head norm with rotary positions of part of the head, and their gradients in one graph, as a
    block runs them, replayed on new inputs beside eager calls; the two backwards share one workspace."""
    Hq, Hk, D, R = 8, 2, 128, 64
    W = (Hq + 2 * Hk) * D

    def inputs(seed):
        return (synth.normal16((T, W), seed, DEV), synth.normal16((T, W), seed + 1, DEV), _pos(T, seed))

    x, gy, pos = inputs(1)
    w, b = synth.gamma_f32(W, 4, DEV), synth.gamma_f32(W, 5, DEV, mean=0.0)
    wq, wk = _weights(D, Hk, 6, False)
    f = _freq(R)
    size = max(rn.layernorm_bwd_workspace_bytes(T, W), rn.rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D))

    def split(t):
        return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)

    def buffers():
        e = lambda *s: torch.empty(s, device=DEV)
        return dict(y=torch.empty((T, W), dtype=BF16, device=DEV), o=torch.empty((T, W), dtype=BF16, device=DEV),
                    dy=torch.zeros((T, W), dtype=BF16, device=DEV), dx=torch.empty((T, W), dtype=BF16, device=DEV),
                    mean=e(T), rstd=e(T), rq=e(T, Hq), rk=e(T, Hk), dw=e(W), db=e(W), dwq=e(D), dwk=e(D),
                    ws=torch.empty(size, dtype=torch.uint8, device=DEV))

    def block(x, gy, pos, o):
        rn.layernorm_fwd(x, w, b, o["y"], o["mean"], o["rstd"], 1e-5)
        q, k = split(o["y"])
        rn.rmsnorm_rope_fwd(q, k, wq, wk, f, *split(o["o"]), o["rq"], o["rk"], pos, 1.0, False, EPS)
        rn.rmsnorm_rope_bwd(*split(gy), q, k, wq, wk, f, o["rq"], o["rk"], *split(o["dy"]), o["dwq"], o["dwk"],
                            o["ws"], pos)
        rn.layernorm_bwd(o["dy"], x, w, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], o["ws"])

    eager, held = buffers(), buffers()
    block(x, gy, pos, held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, gy, pos, held)
    for seed in (11, 22, 33):
        nx, ng, npos = inputs(seed)
        x.copy_(nx), gy.copy_(ng), pos.copy_(npos)
        graph.replay()
        block(nx, ng, npos, eager)
        torch.cuda.synchronize()
        for name in ("y", "dx", "dy"):
            assert torch.equal(_bits(held[name]), _bits(eager[name])), name
        for name in ("mean", "rstd", "rq", "rk", "dw", "db", "dwq", "dwk"):
            assert torch.equal(held[name], eager[name]), name
        # against the definition, gradient by gradient
        dy = torch.zeros((T, W), dtype=torch.float64, device=DEV)
        for g, xx, ww, r, dw, lo, hi in ((*[split(t)[0] for t in (ng, eager["y"])], wq, eager["rq"], "dwq", 0, Hq * D),
                                         (*[split(t)[1] for t in (ng, eager["y"])], wk, eager["rk"], "dwk", Hq * D,
                                          (Hq + Hk) * D)):
            (d, rw), (e, ew) = ref.norm_turn_bwd(g.double(), xx.double(), ww.double(), r.double(), npos, f, 1.0, False)
            ref.assert_within(dw, eager[dw], rw, ew)
            ref.assert_within("dy", eager["dy"][:, lo:hi], d.reshape(T, -1), e.reshape(T, -1), BF16)
        (dx, rdw, rdb), (edx, edw, edb) = ref.ln_bwd(eager["dy"].double(), nx.double(), w.double(),
                                                     eager["mean"].double(), eager["rstd"].double())
        ref.assert_within("dx", eager["dx"], dx, edx, BF16)
        ref.assert_within("dw", eager["dw"], rdw, edw)
        ref.assert_within("db", eager["db"], rdb, edb)
    assert rn.rmsnorm_device_error() == 0


def test_on_a_stream_of_its_own():
    q, k = _heads(1000, 8, 2, 128, 81)
    f = _freq(128)
    o0, k0, o1, k1 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k)
    rn.rope_fwd(q, k, f, o0, k0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rn.rope_fwd(q, k, f, o1, k1, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(_bits(o0), _bits(o1)) and torch.equal(_bits(k0), _bits(k1))


def test_infinity_beside_the_turned_part():
    """An infinite value whose 16-byte vector also holds turned pairs touches its own place alone: its head's
    inverse RMS is zero, so the others are zeros, and its own place is NaN."""
    q, _ = _heads(3, 2, 0, 128, 91)
    q[1, 0, 7] = float("inf")
    w, _ = _weights(128, 0, 92, False)
    for R, inter in ((6, True), (2, True), (6, False)):
        (_, o, r), _ = _norm_fwd(q, None, w, None, _freq(R), None, inter)
        assert float(r[1, 0]) == 0.0
        want = torch.zeros(128, dtype=torch.bool, device=DEV)
        want[7] = True
        assert torch.equal(o[1, 0].isnan(), want) and bool((o[1, 0][~want] == 0).all())
        rest = o.isfinite().all(2)
        rest[1, 0] = True
        assert bool(rest.all())


@pytest.mark.parametrize("size,eps", [(5e17, EPS), (1e16, EPS), (1e14, EPS), (1e-14, 0.0), (1e-18, 0.0)])
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", [(67, 4, 2, 128, 128, False), (67, 4, 2, 256, 64, True), (67, 3, 0, 96, 20, False),
                                               (6001, 4, 1, 64, 64, False)])
def test_norm_and_rope_at_any_magnitude(size, eps, T, Hq, Hk, D, R, inter):
    """Heads whose squares still fit fp32: the inverse RMS to its third power would not."""
    q, k = _heads(T, Hq, Hk, D, 141)
    q, k = q * size, None if k is None else k * size
    g, h = _heads(T, Hq, Hk, D, 142)
    wq, wk = _weights(D, Hk, 143, False)
    pos, f = _pos(T, 144), _freq(R)
    rq, rk = torch.empty((T, Hq), device=DEV), torch.empty((T, Hk), device=DEV) if Hk else None
    oq, ok = torch.empty_like(q), None if k is None else torch.empty_like(k)
    rn.rmsnorm_rope_fwd(q, k, wq, wk, f, oq, ok, rq, rk, pos, SCALE, inter, eps)
    (_, dq, dwq), (_, dk, dwk) = _norm_bwd(g, h, q, k, wq, wk, f, rq, rk, pos, inter)
    eps32 = float(torch.tensor(eps, dtype=torch.float32))
    for name, gg, x, w, o, r, d, dw in (("q", g, q, wq, oq, rq, dq, dwq), ("k", h, k, wk, ok, rk, dk, dwk)):
        if x is None:
            continue
        (want, rstd), (e, er) = ref.norm_turn_fwd(x.double(), w.double(), eps32, pos, f, SCALE, inter)
        ref.assert_within(f"rstd {name}", r, rstd, er)
        ref.assert_within(name, o, want, e, BF16)
        (want, rdw), (e, ew) = ref.norm_turn_bwd(gg.double(), x.double(), w.double(), r.double(), pos, f, SCALE, inter)
        ref.assert_within(f"d{name}", d, want, e, BF16)
        ref.assert_within(f"dw{name}", dw, rdw, ew)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [16, 6001])
@pytest.mark.parametrize("dtype,scale", [(BF16, 1.0), (F16, 2.0 ** 14)])
def test_small_angles_keep_their_digits(T, interleaved, dtype, scale):
    """Pairs (1, 0) at slow frequencies: the sine is right relative to itself, not to the pair. TURN bounds the
    arithmetic; the frequency's rounding is |a| 2^-51 and |p| 2^-62 of an angle, and 2^-55 turns of the phase are kept."""
    turn = 6.283185307179586476925
    n = 37
    f = turn * 1.37 * 2.0 ** -torch.arange(4, 4 + n, device=DEV, dtype=torch.float64)
    pos = torch.tensor([1, -1, 2, 3, -3, 7, 100, -1000, 4095, 0, 65537, 1 << 20, -(1 << 20) - 1, 5, 6, 12345],
                       device=DEV).repeat(T // 16 + 1)[:T]
    x = torch.zeros((T, 1, 80), dtype=dtype, device=DEV)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x[..., first] = 1.0
    a = pos.double()[:, None] * f
    err = a.abs() * 2.0 ** -51 + pos.double().abs()[:, None] * 2.0 ** -62 + turn * 2.0 ** -55
    for back in (False, True):
        o = torch.empty_like(x)
        (rn.rope_bwd if back else rn.rope_fwd)(x, None, f, o, None, pos, scale, interleaved)
        for name, got, want in (("cos", o[:, 0, first], a.cos()), ("sin", o[:, 0, second], -a.sin() if back else a.sin())):
            ref.assert_within(name, got, scale * want, scale * (ref.TURN * want.abs() + err), dtype)


def test_negative_frequencies_at_far_positions():
    """They keep as many digits as positive ones: the angle's error is |a| 2^-51 and |p| 2^-62."""
    turn = 6.283185307179586476925
    f = -turn * torch.tensor([1.1, 1.3, 1.5, 1.7], dtype=torch.float64, device=DEV) * 2.0 ** -30
    pos = torch.tensor([1 << 44, (1 << 44) + 12345, -(1 << 43) - 1, 1 << 40, 10 ** 12 + 7, 1 << 31], device=DEV)
    x = torch.zeros((6, 1, 8), dtype=F16, device=DEV)
    x[..., 0:4] = 1.0
    o = torch.empty_like(x)
    rn.rope_fwd(x, None, f, o, None, pos)
    a = pos.double()[:, None] * f
    err = ref.TURN + a.abs() * 2.0 ** -51 + pos.double().abs()[:, None] * 2.0 ** -62
    ref.assert_within("cos", o[:, 0, 0:4], a.cos(), err, F16)
    ref.assert_within("sin", o[:, 0, 4:8], a.sin(), err, F16)


def test_weight_gradients_of_one_sign_and_many_rows():
    """Sums of products of one sign, longer a lane than any other test's: 38 million rows of 8 values are
    T H / (304 CTAs x 8 warps x 8 groups) = 2000 additions a lane, then 64 groups, 3 partial rows a range, 16 ranges
    and 8 parts."""
    T, H, D = 2432000, 16, 8
    q = synth.normal16((T, H, D), 151, DEV).abs_().add_(0.5)
    g = synth.normal16((T, H, D), 152, DEV).abs_().add_(0.5)
    w = torch.ones(D, device=DEV)
    pos, f = torch.zeros(T, dtype=torch.int64, device=DEV), _freq(2)
    (_, _, r), _ = _norm_fwd(q, None, w, None, f, pos)
    (_, _, dw), _ = _norm_bwd(g, None, q, None, w, None, f, r, None, pos)
    want = torch.zeros(D, dtype=torch.float64, device=DEV)
    for i in range(0, T, 76000):
        n = g[i:i + 76000].double() * q[i:i + 76000].double() * r[i:i + 76000].double()[..., None]
        n[..., :2] *= SCALE
        want += n.sum((0, 1))
    chain = -(-T * H // (304 * 8 * 8)) + 1 + 64 + 3 + 16 + 8
    # of a term: the turn (by no angle, scaled), x r, and the fused product
    ref.assert_within("dw", dw, want, (chain * ref.U + ref.TURN + 2 * ref.U) * want)
