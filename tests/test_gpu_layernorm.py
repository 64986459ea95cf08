"""LayerNorm forward and backward on the GPU against its definition in 64 bits
(``tests/block_ref.py``, with the derivation of the bounds)."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests import block_ref as ref
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

EPS = 1e-5
F32_EPS = float(torch.tensor(EPS, dtype=torch.float32))
BF16, F16 = torch.bfloat16, torch.float16


def _rows(t, pad):
    """t with its rows D + pad apart; the gap holds -7."""
    return synth.strided(t, t.shape[1] + pad) if pad else t


def _inputs(T, D, seed, dtype=BF16, shift=0.0, zc=False, pad=0):
    x = _rows((synth.normal16((T, D), seed, DEV).float() * 1.5 + shift).to(dtype), pad)
    g = _rows(synth.normal16((T, D), seed + 1, DEV, dtype=dtype), pad)
    w = synth.gamma_f32(D, seed + 2, DEV, mean=0.0 if zc else 1.0, std=0.2)
    b = synth.gamma_f32(D, seed + 3, DEV, mean=0.0, std=0.5)
    return x, g, w, b


def _out(T, D, dtype, pad):
    base = torch.full((max(T, 1), D + pad), 3.0, dtype=dtype, device=DEV)
    return base, base[:T, :D]


def _fwd(x, w, b, zc=False, pad=0, stream=None):
    T, D = x.shape
    base, y = _out(T, D, x.dtype, pad)
    mean, rstd = torch.full((T,), -1.0, device=DEV), torch.full((T,), -1.0, device=DEV)
    rn.layernorm_fwd(x, w, b, y, mean, rstd, EPS, zc, stream=stream)
    return base, y, mean, rstd


def _bwd(g, x, w, mean, rstd, bias=True, zc=False, pad=0, ws=None):
    T, D = x.shape
    base, dx = _out(T, D, x.dtype, pad)
    dw = torch.full((D,), 5.0, device=DEV)
    db = torch.full((D,), 5.0, device=DEV) if bias else None
    if ws is None:
        ws = torch.full((max(rn.layernorm_bwd_workspace_bytes(T, D) // 4, 4),), float("nan"), device=DEV)
    rn.layernorm_bwd(g, x, w, mean, rstd, dx, dw, db, ws, zc)
    return base, dx, dw, db


def _check(T, D, seed, dtype=BF16, shift=0.0, zc=False, bias=True, pad=0):
    x, g, w, b = _inputs(T, D, seed, dtype, shift, zc, pad)
    b = b if bias else None
    we = ref.effective(w, zc)
    base, y, mean, rstd = _fwd(x, w, b, zc, pad)
    (ry, rm, rr), (ey, em, er) = ref.ln_fwd(x.double(), we, None if b is None else b.double(), F32_EPS)
    ref.assert_within("mean", mean, rm, em)
    ref.assert_within("rstd", rstd, rr, er)
    ref.assert_within("y", y, ry, ey, dtype)
    gbase, dx, dw, db = _bwd(g, x, w, mean, rstd, bias, zc, pad)
    (rdx, rdw, rdb), (edx, edw, edb) = ref.ln_bwd(g.double(), x.double(), we, mean.double(), rstd.double())
    ref.assert_within("dx", dx, rdx, edx, dtype)
    ref.assert_within("dw", dw, rdw, edw)
    if bias:
        ref.assert_within("db", db, rdb, edb)
    for t in (base, gbase):  # nothing beside the rows was written
        assert bool((t[:, D:] == 3.0).all())


# widths on both sides of every launch shape, a row and a few, odd counts
WIDTHS = [8, 16, 24, 32, 40, 64, 72, 96, 104, 128, 136, 192, 200, 256, 264, 384, 392, 512, 520, 768, 776, 1016, 1024,
          1032, 1280, 1536, 1792, 2048, 2056, 2560, 2568, 3584, 4096, 4104, 5000, 5120, 5128, 6144, 6152, 7168, 8192, 8200,
          10240, 12288, 12296, 14336, 14344, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T,dtype,bias,zc,pad", [(1, BF16, True, False, 0), (37, F16, True, True, 8),
                                                 (131, BF16, False, False, 24)])
def test_against_the_definition(D, T, dtype, bias, zc, pad):
    _check(T, D, seed=D + T, dtype=dtype, bias=bias, zc=zc, pad=pad)


@pytest.mark.parametrize("T,D", [(4099, 5000), (20000, 128), (2500, 4096), (9001, 256), (1500, 16384), (40000, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_rows(T, D, dtype):
    _check(T, D, seed=T, dtype=dtype, zc=dtype == F16, bias=T % 2 == 0)


@pytest.mark.parametrize("D", [64, 4096, 16384])
@pytest.mark.parametrize("shift", [30.0, 300.0])
def test_a_mean_far_from_zero_costs_no_digits(D, shift):
    _check(33, D, seed=7, dtype=F16, shift=shift)


def test_constant_rows():
    """No variance: rstd = eps^-1/2 exactly, n = 0, y = b; dx sums to zero."""
    for D in (128, 4096):
        x = torch.full((5, D), 2.0, dtype=BF16, device=DEV)
        w = synth.gamma_f32(D, 1, DEV)
        b = synth.gamma_f32(D, 2, DEV, mean=0.0)
        _, y, mean, rstd = _fwd(x, w, b)
        assert bool((mean == 2.0).all())
        ref.assert_within("rstd", rstd, torch.full((5,), F32_EPS ** -0.5, device=DEV).double(),
                          torch.full((5,), F32_EPS ** -0.5 * 2 ** -21, device=DEV).double())
        assert torch.equal(y, b.to(BF16).expand(5, D))


@pytest.mark.parametrize("D", [128, 1000, 4096, 16384])
def test_rows_do_not_touch_each_other(D):
    """A row's bits are its own: the same in any batch, at any place and stride, beside rows of NaN and infinity."""
    x0, g0, w, b = _inputs(1, D, 11)
    _, y1, m1, r1 = _fwd(x0, w, b)
    _, dx1, _, _ = _bwd(g0, x0, w, m1, r1)
    for T, at in ((2, 1), (17, 0), (130, 77), (1025, 1024)):
        for pad in (0, 40):
            x, g, _, _ = _inputs(T, D, 100 + T)
            x[at], g[at] = x0[0], g0[0]
            if T > 2:
                x[(at + 1) % T] = float("nan")
                x[(at + 2) % T, D // 2] = float("inf")
            x, g = _rows(x, pad), _rows(g, pad)
            _, y, m, r = _fwd(x, w, b, pad=pad)
            _, dx, _, _ = _bwd(g, x, w, m, r, pad=pad)
            assert torch.equal(y[at].view(torch.int16), y1[0].view(torch.int16))
            assert m[at] == m1[0] and r[at] == r1[0]
            assert torch.equal(dx[at].view(torch.int16), dx1[0].view(torch.int16))


def test_nan_and_infinity_stay_in_their_row_and_column_sums():
    x, g, w, b = _inputs(9, 256, 5)
    x[3, 10] = float("inf")
    x[5, 20] = float("nan")
    _, y, mean, rstd = _fwd(x, w, b)
    bad = torch.zeros(9, dtype=torch.bool, device=DEV)
    bad[3] = bad[5] = True
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isfinite().all(1), ~bad)
    _, dx, dw, db = _bwd(g, x, w, mean, rstd)
    assert torch.equal(dx.isfinite().all(1), ~bad)
    assert bool(dw.isnan().all()) and bool(db.isfinite().all())  # dw takes n of every row, db the gradients alone


@pytest.mark.parametrize("T,D", [(3000, 128), (1111, 4096), (700, 16384)])
def test_weight_gradients_are_the_same_from_run_to_run(T, D):
    x, g, w, b = _inputs(T, D, 21)
    _, _, mean, rstd = _fwd(x, w, b)
    first = _bwd(g, x, w, mean, rstd)
    for _ in range(3):
        again = _bwd(g, x, w, mean, rstd)
        assert torch.equal(first[2], again[2]) and torch.equal(first[3], again[3])
        assert torch.equal(first[1].view(torch.int16), again[1].view(torch.int16))


@pytest.mark.parametrize("T,D", [(300, 96), (300, 520), (200, 4096), (100, 12296)])
def test_the_bias_gradient_changes_nothing_else(T, D):
    x, g, w, b = _inputs(T, D, 25)
    _, _, mean, rstd = _fwd(x, w, b)
    _, dx, dw, _ = _bwd(g, x, w, mean, rstd)
    _, dx2, dw2, _ = _bwd(g, x, w, mean, rstd, bias=False)
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16)) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,D", [((1 << 31) // 16384 + 3, 16384), ((1 << 31) // 128 + 5, 128)])
def test_rows_beyond_two_to_the_31_values(T, D):
    """The last rows of a tensor of more than 2^31 values, against the same rows on their own."""
    x = torch.zeros((T, D), dtype=BF16, device=DEV)
    g = torch.zeros((T, D), dtype=BF16, device=DEV)
    tx, tg, w, b = _inputs(4, D, 61)
    x[-4:], g[-4:] = tx, tg
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    dw, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(rn.layernorm_bwd_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    rn.layernorm_fwd(x, w, b, y, mean, rstd, EPS)
    rn.layernorm_bwd(g, x, w, mean, rstd, dx, dw, db, ws)
    _, ty, tm, tr = _fwd(tx, w, b)
    _, tdx, tdw, tdb = _bwd(tg, tx, w, tm, tr)
    assert torch.equal(y[-4:].view(torch.int16), ty.view(torch.int16)) and torch.equal(rstd[-4:], tr)
    assert torch.equal(dx[-4:].view(torch.int16), tdx.view(torch.int16))
    # the rows of zeros add zeros: the sums are those of four rows in some order
    n = (tx.double() - tm.double()[:, None]) * tr.double()[:, None]
    ref.assert_within("dw", dw, (tg.double() * n).sum(0), 8 * ref.U * (tg.double() * n).abs().sum(0))
    ref.assert_within("db", db, tg.double().sum(0), 8 * ref.U * tg.double().abs().sum(0))


def test_the_binding_refuses_what_would_be_read_wrongly():
    x, g, w, b = _inputs(8, 128, 71)
    y, m, r = torch.empty_like(x), torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    for bad in (dict(w=w.half()), dict(w=w.cpu()), dict(w=w[:64]), dict(w=w.repeat(2)[::2]), dict(b=b.double()),
                dict(y=y.half()), dict(y=y.cpu()), dict(mean=m[:4]), dict(rstd=r.half())):
        a = {**dict(w=w, b=b, y=y, mean=m, rstd=r), **bad}
        with pytest.raises(TypeError):
            rn.layernorm_fwd(x, a["w"], a["b"], a["y"], a["mean"], a["rstd"])
    with pytest.raises(ValueError):
        rn.layernorm_fwd(x, w, b, y[:4], m, r)
    with pytest.raises(ValueError):
        rn.layernorm_fwd(x.t().contiguous().t(), w, b, y, m, r)
    with pytest.raises(TypeError):
        rn.layernorm_fwd(x.float(), w, b, y, m, r)
    with pytest.raises(rn.RmsNormError, match="EALIGN"):
        rn.layernorm_fwd(x, torch.empty(129, device=DEV)[1:], b, y, m, r)


def test_the_entry_points_called_with_their_own_arguments():
    """The C entry points, which the binding calls with an array, argument by argument: the same bits."""
    lib, st = rn.load(), torch.cuda.current_stream().cuda_stream
    T, D = 21, 200
    x, g = (synth.normal16((T, D), i, DEV) for i in (131, 132))
    w, b = synth.gamma_f32(D, 133, DEV), synth.gamma_f32(D, 134, DEV, mean=0.0)
    out = []
    for direct in (False, True):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        m, r = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        dw, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        ws = torch.empty(rn.layernorm_bwd_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
        if direct:
            assert lib.layernorm_fwd(x.data_ptr(), D, w.data_ptr(), b.data_ptr(), y.data_ptr(), D, m.data_ptr(),
                                     r.data_ptr(), T, D, 1e-5, 1, 0, st) == 0
            assert lib.layernorm_bwd(g.data_ptr(), D, x.data_ptr(), D, w.data_ptr(), m.data_ptr(), r.data_ptr(),
                                     dx.data_ptr(), D, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), T, D, 1, 0,
                                     st) == 0
        else:
            rn.layernorm_fwd(x, w, b, y, m, r, 1e-5, True)
            rn.layernorm_bwd(g, x, w, m, r, dx, dw, db, ws, True)
        out.append((y, dx, m, r, dw, db))
    for a, c in zip(*out):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_no_rows():
    x, g, w, b = _inputs(0, 128, 1)
    _fwd(x, w, b)
    e = torch.empty(0, device=DEV)
    _, _, dw, db = _bwd(g, x, w, e, e)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_workspace_queries():
    """One workspace of the largest size serves every smaller T, a byte less is refused."""
    T_max, D = 5000, 512
    most = rn.layernorm_bwd_workspace_bytes_max(T_max, D)
    sizes = [rn.layernorm_bwd_workspace_bytes(t, D) for t in range(1, T_max + 1)]
    assert max(sizes) <= most
    x, g, w, b = _inputs(300, D, 3)
    _, _, mean, rstd = _fwd(x, w, b)
    ws = torch.empty(most, dtype=torch.uint8, device=DEV)
    _bwd(g, x, w, mean, rstd, ws=ws)
    need = rn.layernorm_bwd_workspace_bytes(300, D)
    with pytest.raises(rn.RmsNormError, match="EWORKSPACE"):
        _bwd(g, x, w, mean, rstd, ws=ws[:need - 16])


@pytest.mark.parametrize("T,D", [(900, 4096), (3000, 128), (300, 12296)])
def test_captured_and_replayed(T, D):
    """Forward and backward in a graph, replayed on new inputs, beside eager calls with a workspace of their own."""
    x, g, w, b = _inputs(T, D, 31)
    _fwd(x, w, b)  # the library's launch caches exist before the capture
    warm = _fwd(x, w, b)
    _bwd(g, x, w, warm[2], warm[3])
    torch.cuda.synchronize()
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(rn.layernorm_bwd_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rn.layernorm_fwd(x, w, b, y, mean, rstd, EPS)
        rn.layernorm_bwd(g, x, w, mean, rstd, dx, dw, db, ws)
    for seed in (41, 42):
        nx, ng, _, _ = _inputs(T, D, seed)
        x.copy_(nx)
        g.copy_(ng)
        graph.replay()
        _, ey, em, er = _fwd(nx, w, b)
        _, edx, edw, edb = _bwd(ng, nx, w, em, er)
        torch.cuda.synchronize()
        for a, c in ((y, ey), (dx, edx)):
            assert torch.equal(a.view(torch.int16), c.view(torch.int16))
        for a, c in ((mean, em), (rstd, er), (dw, edw), (db, edb)):
            assert torch.equal(a, c)


def test_on_a_stream_of_its_own():
    x, g, w, b = _inputs(2000, 1024, 51)
    _, y0, _, _ = _fwd(x, w, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, y1, _, _ = _fwd(x, w, b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y0.view(torch.int16), y1.view(torch.int16))
    assert rn.rmsnorm_device_error() == 0


def test_shapes_are_named_in_refusals():
    x, g, w, b = _inputs(8, 128, 71)
    m, r, dw = torch.empty(8, device=DEV), torch.empty(8, device=DEV), torch.empty(128, device=DEV)
    for t in (x.view(2, 4, 128), x[0]):
        with pytest.raises(TypeError, match="x: expected a 2-D"):
            rn.layernorm_fwd(t, w, b, torch.empty_like(t), m, r)
        with pytest.raises(TypeError, match="x: expected a 2-D"):
            rn.layernorm_bwd(t, t, w, m, r, torch.empty_like(t), dw, None, torch.empty(8192, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError, match="y: expected a 2-D"):
        rn.layernorm_fwd(x, w, b, x.view(2, 4, 128), m, r)


def test_the_stride_of_a_single_row_is_never_taken():
    _, _, w, b = _inputs(8, 128, 71)
    m, r, dw = torch.empty(8, device=DEV), torch.empty(8, device=DEV), torch.empty(128, device=DEV)
    wide = synth.normal16((1, 132), 5, DEV)  # rows 132 apart: of one row, a stride that is never taken
    x1, y0, y1 = wide[:, :128], torch.empty((1, 128), dtype=BF16, device=DEV), torch.empty_like(wide)[:, :128]
    rn.layernorm_fwd(x1.contiguous(), w, b, y0, m[:1], r[:1])
    m1, r1 = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    rn.layernorm_fwd(x1, w, b, y1, m1, r1)
    assert torch.equal(y0, y1) and torch.equal(m1, m[:1]) and torch.equal(r1, r[:1])
    ws = torch.empty(rn.layernorm_bwd_workspace_bytes(1, 128), dtype=torch.uint8, device=DEV)
    d0, d1 = torch.empty_like(y0), torch.empty_like(wide)[:, :128]
    rn.layernorm_bwd(x1.contiguous(), x1.contiguous(), w, m1, r1, d0, dw, None, ws)
    rn.layernorm_bwd(x1, x1, w, m1, r1, d1, dw, None, ws)
    assert torch.equal(d0, d1)
    with pytest.raises(rn.RmsNormError, match="EALIGN"):
        two = synth.normal16((2, 132), 5, DEV)[:, :128]
        rn.layernorm_fwd(two, w, b, torch.empty((2, 128), dtype=BF16, device=DEV), m[:2], r[:2])


@pytest.mark.parametrize("T,D", [(20011, 1024), (9001, 1536), (20000, 2048), (6007, 3080), (30001, 520), (20000, 776),
                                 (6001, 4104), (3001, 6152)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rings_and_rows_go_round(T, D, dtype):
    """More rows a team than its ring has stages, or than one trip of the forward's loop, and an uneven last chunk."""
    _check(T, D, seed=T + D, dtype=dtype, zc=dtype == F16, bias=T % 2 == 1)


@pytest.mark.parametrize("D", [24, 1000, 1016, 5000, 16376])
@pytest.mark.parametrize("value", [2.0, -1.171875, 3.0078125, 1.3e30])
def test_constant_rows_at_widths_that_are_no_power_of_two(D, value):
    """The mean is the sum's correctly rounded quotient by D, where 1 / D is not exact: n = 0 and y = b."""
    x = torch.full((5, D), value, dtype=BF16, device=DEV)
    w, b = synth.gamma_f32(D, 1, DEV), synth.gamma_f32(D, 2, DEV, mean=0.0)
    _, y, mean, rstd = _fwd(x, w, b)
    assert bool((mean == x[:, 0].float()).all())
    assert torch.equal(y, b.to(BF16).expand(5, D))


@pytest.mark.parametrize("size,eps", [(1e17, 1e-5), (1e14, 1e-5), (1e-14, 0.0), (1e-18, 0.0)])
@pytest.mark.parametrize("T,D", [(67, 128), (67, 1000), (67, 2048), (67, 5000), (67, 16384)])
def test_any_magnitude(size, eps, T, D):
    """Rows whose sum of squares still fits fp32; one that does not (16384 values of 1.5e17: 3.7e38) has rstd 0."""
    x, g, w, b = _inputs(T, D, 161)
    x = x * size
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (T, T, D, D))
    ws = torch.empty(rn.layernorm_bwd_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    rn.layernorm_fwd(x, w, b, y, mean, rstd, eps)
    if D * (1.5 * size) ** 2 > 3.5e38:
        assert bool((rstd == 0).all()) and torch.equal(y, b.to(BF16).expand(T, D))
        return
    rn.layernorm_bwd(g, x, w, mean, rstd, dx, dw, db, ws)
    (ry, rm, rr), (ey, em, er) = ref.ln_fwd(x.double(), w.double(), b.double(), float(torch.tensor(eps, dtype=torch.float32)))
    ref.assert_within("mean", mean, rm, em)
    ref.assert_within("rstd", rstd, rr, er)
    ref.assert_within("y", y, ry, ey, BF16)
    (rdx, rdw, rdb), (edx, edw, edb) = ref.ln_bwd(g.double(), x.double(), w.double(), mean.double(), rstd.double())
    ref.assert_within("dx", dx, rdx, edx, BF16)
    ref.assert_within("dw", dw, rdw, edw)
    ref.assert_within("db", db, rdb, edb)


def test_weight_gradients_of_one_sign_and_many_rows():
    """Sums of terms of one sign along the longest chains that the chunks allow: 256 rows a lane, 256 groups of a CTA,
    3 partial rows a range, 16 ranges and 8 parts."""
    T, D = 304 * 256 * 256, 8
    x = synth.normal16((T, D), 171, DEV)
    g = synth.normal16((T, D), 172, DEV).abs_().add_(0.5)
    w = torch.ones(D, device=DEV)
    _, _, mean, rstd = _fwd(x, w, None)
    # the sign of n = (x - mean) rstd on g: every product is positive
    g = torch.where(x.float() < mean[:, None], -g, g)
    _, _, dw, db = _bwd(g, x, w, mean, rstd)
    want, size, sums = (torch.zeros(D, dtype=torch.float64, device=DEV) for _ in range(3))
    for i in range(0, T, 1 << 18):
        gg = g[i:i + (1 << 18)].double()
        n = (x[i:i + (1 << 18)].double() - mean[i:i + (1 << 18), None].double()) * rstd[i:i + (1 << 18), None].double()
        want += (gg * n).sum(0)
        sums += gg.sum(0)
        size += gg.abs().sum(0)
    chain = 256 + 256 + 3 + 16 + 8
    ref.assert_within("dw", dw, want, (chain + 4) * ref.U * want.abs())
    ref.assert_within("db", db, sums, chain * ref.U * size)
