"""Projections and gated feed-forward blocks on the GPU against their definitions
in 64 bits (``tests/linear_ref.py``), their refusals, streams and graphs."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests import linear_ref as ref
from tests.block_ref import assert_within
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
ACTS = sorted(rn.LINEAR_ACTS)


def _bits(t):
    return t.contiguous().view(torch.int16)


def _mat(rows, cols, seed, dtype=BF16, std=1.0, pad=0, beside=float("nan")):
    """A matrix of normal values, its rows ``cols + pad`` apart with ``beside`` between them."""
    base = torch.full((rows, cols + pad), beside, dtype=dtype, device=DEV)
    base[:, :cols] = (synth.normal16((rows, cols), seed, DEV, dtype=torch.float16).float() * std).to(dtype)
    return base[:, :cols]


def _out(rows, cols, dtype=BF16, pad=0):
    base = torch.full((rows + 2, cols + pad), 3.0, dtype=dtype, device=DEV)
    return base, base[1:rows + 1, :cols]


def _untouched(base, out):
    keep = torch.ones(base.shape, dtype=torch.bool, device=DEV)
    keep[1:out.shape[0] + 1, :out.shape[1]] = False
    assert bool((base[keep] == 3.0).all())


def _ws(n):
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)  # NaNs in every format


def _d(t):
    return None if t is None else t.double()


# T: every count of rows a CTA copies, products of 64 and of 128 rows, several row tiles, pairs of CTAs
SIZES = [(1, 8, 8), (2, 64, 32), (3, 72, 40), (8, 4096, 264), (9, 16, 2056), (63, 200, 104), (64, 136, 1000), (65, 128, 64),
         (113, 1000, 200), (120, 64, 48), (121, 72, 512), (128, 256, 96), (129, 520, 80), (257, 40, 136), (300, 1000, 264),
         (1021, 104, 2056), (2309, 192, 1160)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,act,bias,res,save,pad", [(BF16, "none", False, False, False, 0), (F16, "gelu", True, True, True, 8),
                                                         (BF16, "silu", True, False, True, 64), (F16, "none", False, True, False, 24)])
def test_linear_fwd(T, K, N, dtype, act, bias, res, save, pad):
    x, w = _mat(T, K, T + K, dtype, pad=pad), _mat(N, K, T + N, dtype, K ** -0.5, pad)
    b = synth.gamma_f32(N, 3, DEV, mean=0.0, std=0.5) if bias else None
    r = _mat(T, N, 5, dtype, pad=pad) if res else None
    by, y = _out(T, N, dtype, pad)
    bz, z = _out(T, N, dtype, 8) if save else (None, None)
    rn.linear_fwd(x, w, b, r, y, z, act)
    (wy, wz), (ey, ez) = ref.linear_fwd(_d(x), _d(w), _d(b), _d(r), act)
    assert_within("y", y, wy, ey, dtype)
    _untouched(by, y)
    if save:
        assert_within("z", z, wz, ez, dtype)
        _untouched(bz, z)
    assert rn.rmsnorm_device_error() == 0


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,act,bias,pad", [(BF16, "none", True, 0), (F16, "gelu_tanh", True, 8), (BF16, "gelu", False, 64)])
def test_linear_bwd(T, K, N, dtype, act, bias, pad):
    x, w, g = _mat(T, K, T + K, dtype, pad=pad), _mat(N, K, T + N, dtype, K ** -0.5, pad), _mat(T, N, 7, dtype, 0.25, pad)
    z = _mat(T, N, 9, dtype, 1.5, 16) if act != "none" else None
    (bx, dx), (bw, dw) = _out(T, K, dtype, pad), _out(N, K, dtype, 8)
    db = torch.full((N,), 3.0, device=DEV) if bias else None
    rn.linear_bwd(g, x, w, z, dx, dw, db, _ws(rn.linear_bwd_workspace_bytes(T, N, K, act)), act)
    (wx, ww, wb), (ex, ew, eb) = ref.linear_bwd(_d(g), _d(x), _d(w), _d(z), act, dtype)
    assert_within("dx", dx, wx, ex, dtype)
    assert_within("dw", dw, ww, ew, dtype)
    if bias:
        assert_within("db", db, wb, eb)
    _untouched(bx, dx)
    _untouched(bw, dw)


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,act,save,pad", [(BF16, "silu", False, 0), (F16, "gelu", True, 8), (BF16, "relu", True, 64)])
def test_gated_fwd(T, K, N, dtype, act, save, pad):
    x = _mat(T, K, T + K, dtype, pad=pad)
    wg, wu = _mat(N, K, T + N, dtype, K ** -0.5, pad), _mat(N, K, T + N + 1, dtype, K ** -0.5, 8)
    bh, h = _out(T, N, dtype, pad)
    (bg, gate), (bu, up) = (_out(T, N, dtype, 8), _out(T, N, dtype)) if save else ((None, None), (None, None))
    rn.linear_gated_fwd(x, wg, wu, h, gate, up, act)
    want, err = ref.gated_fwd(_d(x), _d(wg), _d(wu), act)
    for name, base, o, v, e in zip(("h", "gate", "up"), (bh, bg, bu), (h, gate, up), want, err):
        if o is not None:
            assert_within(name, o, v, e, dtype)
            _untouched(base, o)


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,act,pad", [(BF16, "silu", 0), (F16, "gelu_tanh", 8), (BF16, "sigmoid", 64)])
def test_gated_bwd(T, K, N, dtype, act, pad):
    x, g = _mat(T, K, T + K, dtype, pad=pad), _mat(T, N, 7, dtype, 0.25, pad)
    wg, wu = _mat(N, K, T + N, dtype, K ** -0.5, pad), _mat(N, K, T + N + 1, dtype, K ** -0.5, 8)
    gate, up = _mat(T, N, 9, dtype, 1.5, 16), _mat(T, N, 10, dtype, 1.0, pad)
    outs = [_out(T, K, dtype, pad), _out(N, K, dtype, 8), _out(N, K, dtype)]
    rn.linear_gated_bwd(g, x, wg, wu, gate, up, *(o for _, o in outs), _ws(rn.linear_gated_bwd_workspace_bytes(T, N, K)), act)
    want, err = ref.gated_bwd(_d(g), _d(x), _d(wg), _d(wu), _d(gate), _d(up), act, dtype)
    for name, (base, o), v, e in zip(("dx", "dwg", "dwu"), outs, want, err):
        assert_within(name, o, v, e, dtype)
        _untouched(base, o)


@pytest.mark.parametrize("T,K,N", [(2560, 136, 1032), (700, 264, 4104), (5000, 72, 264), (9000, 264, 136)])
def test_pairs_of_ctas_and_split_weight_gradients(T, K, N):
    test_linear_fwd(T, K, N, BF16, "gelu_tanh", True, True, True, 8)
    test_linear_bwd(T, K, N, BF16, "silu", True, 8)
    test_gated_fwd(T, K, N, F16, "silu", True, 8)
    test_gated_bwd(T, K, N, F16, "silu", 8)


@pytest.mark.parametrize("T,K,N", [(4864, 1000, 1024), (4864, 1024, 1000), (600, 1024, 4864), (4864, 1024, 520), (4860, 200, 512)])
def test_the_largest_tiles(T, K, N):
    """Sizes whose outputs are whole waves of 256 x 256 tiles: forward, input gradient, weight gradient, and gated."""
    test_linear_fwd(T, K, N, F16, "silu", True, True, True, 8)
    test_linear_bwd(T, K, N, F16, "none", True, 8)
    test_gated_fwd(T, K, N, BF16, "gelu", True, 8)
    test_gated_bwd(T, K, N, BF16, "silu", 8)


# --------------------------------------------------------------------------
# activations over their whole range
# --------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_activations_of_every_size(act, dtype):
    """z is x's first value itself: values of every size, signed zeros among them."""
    top = 60000.0 if dtype == F16 else 3e38
    z = torch.cat((torch.linspace(-24, 24, 1537), torch.logspace(-30, 2, 200), -torch.logspace(-30, 2, 200),
                   torch.tensor([0.0, -0.0, 200.0, -200.0, top, -top]))).to(DEV).to(dtype)
    T = z.numel()
    x = torch.zeros((T, 8), dtype=dtype, device=DEV)
    x[:, 0] = z
    w = torch.zeros((8, 8), dtype=dtype, device=DEV)
    w[:, 0] = 1.0
    y = torch.empty((T, 8), dtype=dtype, device=DEV)
    rn.linear_fwd(x, w, None, None, y, None, act)
    (a, s), (ea, es) = ref.act(act, z.double())
    assert_within("value", y, a[:, None].expand(T, 8), ea[:, None], dtype)
    # the slopes, through db of single rows: g = 1 at its own row's column
    g = torch.zeros((T, T + (-T) % 8), dtype=dtype, device=DEV)
    g[:, :T].fill_diagonal_(1.0)
    zz = torch.zeros_like(g)
    zz[:, :T] = z[:, None]
    db = torch.empty(g.shape[1], device=DEV)
    ws = _ws(rn.linear_bwd_workspace_bytes(T, g.shape[1], 8, act))
    rn.linear_bwd(g, x, torch.zeros((g.shape[1], 8), dtype=dtype, device=DEV), zz, None, None, db, ws, act)
    assert_within("slope", db[:T], s, es + 4 * 2.0 ** -24 * s.abs())


def test_nan_and_infinity_stay_in_their_row():
    T, K, N = 200, 136, 264
    x, w = _mat(T, K, 1), _mat(N, K, 2, std=0.1)
    x[7, 3], x[150, 135], x[199, 0] = float("nan"), float("inf"), float("-inf")
    for act in ACTS:
        y, h = torch.empty((T, N), dtype=BF16, device=DEV), torch.empty((T, N), dtype=BF16, device=DEV)
        rn.linear_fwd(x, w, None, None, y, None, act)
        rn.linear_gated_fwd(x, w, w, h, None, None, act)
        good = torch.ones(T, dtype=torch.bool, device=DEV)
        good[[7, 150, 199]] = False
        assert bool(y[good].isfinite().all()) and bool(h[good].isfinite().all())
        assert bool(y[7].isnan().all()) and bool(h[7].isnan().all())


# --------------------------------------------------------------------------
# batch invariance
# --------------------------------------------------------------------------
@pytest.mark.parametrize("K,N", [(1000, 2056), (4096, 512), (72, 40)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_do_not_depend_on_the_batch(K, N, dtype):
    T = 4100
    x, g = _mat(T, K, 1, dtype), _mat(T, N, 2, dtype)
    w, v = _mat(N, K, 3, dtype, K ** -0.5), _mat(N, K, 4, dtype, K ** -0.5)
    gate, up = _mat(T, N, 5, dtype), _mat(T, N, 6, dtype)
    b = synth.gamma_f32(N, 7, DEV)

    def step(rows):
        n = len(range(*rows.indices(T)))
        y, z, h, p, q = (torch.empty((n, N), dtype=dtype, device=DEV) for _ in range(5))
        dx, dh = torch.empty((n, K), dtype=dtype, device=DEV), torch.empty((n, K), dtype=dtype, device=DEV)
        rn.linear_fwd(x[rows], w, b, g[rows], y, z, "silu")
        rn.linear_gated_fwd(x[rows], w, v, h, p, q)
        rn.linear_bwd(g[rows], x[rows], w, gate[rows], dx, None, None, _ws(rn.linear_bwd_workspace_bytes(n, N, K, "gelu")), "gelu")
        rn.linear_gated_bwd(g[rows], x[rows], w, v, gate[rows], up[rows], dh, None, None,
                            _ws(rn.linear_gated_bwd_workspace_bytes(n, N, K)))
        return y, z, h, p, q, dx, dh

    whole = step(slice(0, T))
    for n in (1, 5, 16, 17, 63, 64, 65, 100, 120, 121, 128, 129, 200, 257, 300, 500, 800, 1000, 1300, 2000, 2560, 3000, 3900):
        for first in (0, 1234 if n < 2000 else 7, T - n):
            for a, b_ in zip(step(slice(first, first + n)), whole):
                assert torch.equal(_bits(a), _bits(b_[first:first + n])), (n, first)


def test_weight_gradients_repeat_bit_for_bit():
    T, K, N = 3001, 520, 264
    x, g, z = _mat(T, K, 1), _mat(T, N, 2), _mat(T, N, 3)
    w = _mat(N, K, 4)
    outs = []
    for _ in range(3):
        dw, db = torch.empty((N, K), dtype=BF16, device=DEV), torch.empty(N, device=DEV)
        rn.linear_bwd(g, x, w, z, None, dw, db, _ws(rn.linear_bwd_workspace_bytes(T, N, K, "silu")), "silu")
        outs.append((dw, db))
    for dw, db in outs[1:]:
        assert torch.equal(_bits(dw), _bits(outs[0][0])) and torch.equal(db, outs[0][1])


# --------------------------------------------------------------------------
# calls
# --------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 40, 300, 2600])
def test_residual_in_place(T):
    K, N = 264, 1032
    x, w, r = _mat(T, K, 1), _mat(N, K, 2), _mat(T, N, 3, pad=8)
    y = torch.empty((T, N), dtype=BF16, device=DEV)
    rn.linear_fwd(x, w, None, r, y)
    rn.linear_fwd(x, w, None, r, r)
    assert torch.equal(_bits(y), _bits(r))


def test_no_rows():
    K, N = 64, 40
    x, g, w = (torch.empty(s, dtype=BF16, device=DEV) for s in ((0, K), (0, N), (N, K)))
    rn.linear_fwd(x, w, None, None, g)
    rn.linear_gated_fwd(x, w, w, g)
    assert rn.linear_bwd_workspace_bytes(0, N, K) == 0 and rn.linear_gated_bwd_workspace_bytes(0, N, K) == 0
    bw, dw = _out(N, K, pad=8)
    db = torch.full((N,), 3.0, device=DEV)
    rn.linear_bwd(g, x, w, None, x, dw, db, _ws(0))
    assert bool((dw == 0).all()) and bool((db == 0).all())
    _untouched(bw, dw)
    bv, dv = _out(N, K)
    dw.fill_(3.0)
    rn.linear_gated_bwd(g, x, w, w, g, g, None, dw, dv, _ws(0))
    assert bool((dw == 0).all()) and bool((dv == 0).all())
    _untouched(bv, dv)


def test_gradients_one_at_a_time():
    T, K, N = 130, 264, 520
    x, g, w, v, z, u = _mat(T, K, 1), _mat(T, N, 2), _mat(N, K, 3), _mat(N, K, 4), _mat(T, N, 5), _mat(T, N, 6)
    ws = _ws(max(rn.linear_bwd_workspace_bytes(T, N, K, "gelu"), rn.linear_gated_bwd_workspace_bytes(T, N, K)))
    for act in ("none", "gelu"):
        full = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
        rn.linear_bwd(g, x, w, z, *full, ws, act)
        for i in range(3):
            some = [torch.empty_like(t) if j == i else None for j, t in enumerate(full)]
            rn.linear_bwd(g, x, w, z, *some, ws, act)
            assert torch.equal(some[i], full[i])
    full = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    rn.linear_gated_bwd(g, x, w, v, z, u, *full, ws)
    dx, a, b = (torch.empty_like(t) for t in full)
    rn.linear_gated_bwd(g, x, w, v, z, u, dx, None, None, ws)
    rn.linear_gated_bwd(g, x, w, v, z, u, None, a, b, ws)
    assert all(torch.equal(p, q) for p, q in zip((dx, a, b), full))


def test_views_of_wider_matrices():
    """wg and wu as halves of one matrix, x as part of another's columns."""
    T, K, N = 77, 264, 136
    both, wide = _mat(2 * N, K, 1, std=0.1), _mat(T, 3 * K, 2)
    x = wide[:, K:2 * K]
    a, b = (torch.empty((T, N), dtype=BF16, device=DEV) for _ in range(2))
    rn.linear_gated_fwd(x, both[:N], both[N:], a)
    rn.linear_gated_fwd(x.contiguous(), both[:N].clone(), both[N:].clone(), b)
    assert torch.equal(_bits(a), _bits(b))
    row = torch.empty((1, N), dtype=BF16, device=DEV)
    rn.linear_fwd(wide[5:6, K:2 * K], both[:N], None, None, row)
    rn.linear_fwd(x, both[:N], None, None, a)
    assert torch.equal(_bits(row), _bits(a[5:6]))


@pytest.mark.parametrize("T", [1, 100, 2600])
def test_outputs_as_parts_of_wider_matrices(T):
    """gate and up side by side in one buffer, dwg and dwu one above the other, each between columns that stay as they were."""
    K, N = 264, 1032
    x, g, wg, wu = _mat(T, K, 1), _mat(T, N, 2), _mat(N, K, 3, std=0.1), _mat(N, K, 4, std=0.1)
    h, gate, up = (torch.empty((T, N), dtype=BF16, device=DEV) for _ in range(3))
    rn.linear_gated_fwd(x, wg, wu, h, gate, up)
    both = torch.full((T, 2 * N + 24), 3.0, dtype=BF16, device=DEV)
    wide = torch.full((T, N + 16), 3.0, dtype=BF16, device=DEV)
    rn.linear_gated_fwd(x, wg, wu, wide[:, 8:N + 8], both[:, 8:N + 8], both[:, N + 16:2 * N + 16])
    for a, b in ((h, wide[:, 8:N + 8]), (gate, both[:, 8:N + 8]), (up, both[:, N + 16:2 * N + 16])):
        assert torch.equal(_bits(a), _bits(b))
    gaps = torch.cat((wide[:, :8], wide[:, -8:], both[:, :8], both[:, N + 8:N + 16], both[:, -8:]), 1)
    assert bool((gaps == 3.0).all())
    ws = _ws(rn.linear_gated_bwd_workspace_bytes(T, N, K))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    rn.linear_gated_bwd(g, x, wg, wu, gate, up, dx, dwg, dwu, ws)
    stack, dwide = torch.full((2 * N, K + 8), 3.0, dtype=BF16, device=DEV), torch.full((T, K + 8), 3.0, dtype=BF16, device=DEV)
    rn.linear_gated_bwd(g, x, wg, wu, both[:, 8:N + 8], both[:, N + 16:2 * N + 16], dwide[:, 8:], stack[:N, :K], stack[N:, :K], ws)
    for a, b in ((dx, dwide[:, 8:]), (dwg, stack[:N, :K]), (dwu, stack[N:, :K])):
        assert torch.equal(_bits(a), _bits(b))
    assert bool((stack[:, K:] == 3.0).all()) and bool((dwide[:, :8] == 3.0).all())


def test_more_than_two_to_the_31_values():
    T, K, N = (1 << 31) // 16384 + 300, 64, 16384
    x, w = _mat(T, K, 1), _mat(N, K, 2)
    y, few = torch.empty((T, N), dtype=BF16, device=DEV), torch.empty((200, N), dtype=BF16, device=DEV)
    rn.linear_fwd(x, w, None, None, y)
    rn.linear_fwd(x[-200:], w, None, None, few)
    assert torch.equal(_bits(y[-200:]), _bits(few))
    dx, dfew = torch.empty_like(x), torch.empty_like(x[:200])
    ws = _ws(rn.linear_bwd_workspace_bytes(T, N, K, "silu"))
    z = y
    db = torch.empty(N, device=DEV)
    rn.linear_bwd(y, x, w, z, dx, None, db, ws, "silu")
    rn.linear_bwd(y[-200:], x[-200:], w, z[-200:], dfew, None, None, ws, "silu")
    assert torch.equal(_bits(dx[-200:]), _bits(dfew)) and bool(db.isfinite().all())


@pytest.mark.parametrize("T,K,N", [(3, 8, 1 << 20), (3, 1 << 20, 8), (300, 1 << 17, 24), (1 << 20, 8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_longest_sides(T, K, N, dtype):
    """Values of -1, 0 and 1, whose sums are exact in fp32: the results are the rounded integers themselves."""
    def ints(r, c, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        return torch.randint(-1, 2, (r, c), generator=g, device=DEV).to(dtype)

    def same(got, want):
        assert torch.equal(got, want.to(dtype))

    x, w, v, g = ints(T, K, 1), ints(N, K, 2), ints(N, K, 3), ints(T, N, 4)
    y, h = torch.empty_like(g), torch.empty_like(g)
    rn.linear_fwd(x, w, None, g, y)
    rn.linear_gated_fwd(x, w, v, h, None, None, "relu")
    z, u = x.double() @ w.double().t(), x.double() @ v.double().t()
    same(y, z + g.double())
    ok = (z.clamp_min(0) * u).abs() < 2.0 ** 24  # exact there
    assert torch.equal(h[ok], (z.clamp_min(0) * u).to(dtype)[ok])
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
    rn.linear_bwd(g, x, w, None, dx, dw, db, _ws(rn.linear_bwd_workspace_bytes(T, N, K)))
    same(dx, g.double() @ w.double())
    same(dw, g.double().t() @ x.double())
    assert torch.equal(db, g.double().sum(0).float())


def test_long_sums_of_one_sign():
    T, N = 200000, 72
    g = torch.full((T, N), 1.0, dtype=BF16, device=DEV)
    x, w = torch.full((T, 8), 1.0, dtype=BF16, device=DEV), torch.zeros((N, 8), dtype=BF16, device=DEV)
    dw, db = torch.empty_like(w), torch.empty(N, device=DEV)
    rn.linear_bwd(g, x, w, None, None, dw, db, _ws(rn.linear_bwd_workspace_bytes(T, N, 8)))
    assert bool((db == float(T)).all())
    want = torch.tensor(float(T)).to(BF16)
    assert bool((dw.cpu() == want).all())


def _step_buffers(seed, T, K, N):
    m = lambda r, c, i, **kw: _mat(r, c, seed + i, **kw)
    e = lambda r, c: torch.empty((r, c), dtype=BF16, device=DEV)
    return dict(x=m(T, K, 0), g=m(T, K, 1), wg=m(N, K, 2, std=0.1), wu=m(N, K, 3, std=0.1), wd=m(K, N, 4, std=0.1),
                b=synth.gamma_f32(K, seed, DEV), h=e(T, N), gate=e(T, N), up=e(T, N), y=e(T, K), gh=e(T, N), dx=e(T, K),
                dwg=e(N, K), dwu=e(N, K), dwd=e(K, N), db=torch.empty(K, device=DEV),
                ws=_ws(max(rn.linear_gated_bwd_workspace_bytes(T, N, K), rn.linear_bwd_workspace_bytes(T, K, N))))


def _block_step(b):
    """A gated feed-forward block and its gradients."""
    rn.linear_gated_fwd(b["x"], b["wg"], b["wu"], b["h"], b["gate"], b["up"])
    rn.linear_fwd(b["h"], b["wd"], b["b"], b["x"], b["y"])
    rn.linear_bwd(b["g"], b["h"], b["wd"], None, b["gh"], b["dwd"], b["db"], b["ws"])
    rn.linear_gated_bwd(b["gh"], b["x"], b["wg"], b["wu"], b["gate"], b["up"], b["dx"], b["dwg"], b["dwu"], b["ws"])


OUTS = ("h", "gate", "up", "y", "gh", "dx", "dwg", "dwu", "dwd", "db")


def _same(a, b):
    for k in OUTS:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("T,K,N", [(5, 264, 520), (300, 264, 520), (2600, 520, 1032)])
def test_graph_replay_matches_eager(T, K, N):
    b, want = _step_buffers(1, T, K, N), _step_buffers(1, T, K, N)
    _block_step(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        _block_step(b)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        _same(b, want)
    new = _step_buffers(50, T, K, N)
    for k in ("x", "g", "wg", "wu", "wd", "b"):
        b[k].copy_(new[k])
    graph.replay()
    _block_step(new)
    torch.cuda.synchronize()
    _same(b, new)


def test_two_streams_at_once():
    sizes = ((300, 264, 520), (2600, 264, 520))
    alone = [_step_buffers(i, *s) for i, s in enumerate(sizes)]
    for b in alone:
        _block_step(b)
    torch.cuda.synchronize()
    runs = [_step_buffers(i, *s) for i, s in enumerate(sizes)]
    streams = [torch.cuda.Stream(DEV) for _ in runs]
    for _ in range(5):
        for b in runs:
            for k in OUTS:
                b[k].zero_()
        torch.cuda.synchronize()
        for st, b in zip(streams, runs):
            with torch.cuda.stream(st):
                _block_step(b)
        torch.cuda.synchronize()
        for a, b in zip(alone, runs):
            _same(a, b)
    assert rn.rmsnorm_device_error() == 0


def test_the_binding_refuses_what_would_be_read_wrongly():
    T, K, N = 16, 64, 40
    x, w, g = _mat(T, K, 1), _mat(N, K, 2), _mat(T, N, 3)
    y, b, ws = torch.empty_like(g), torch.zeros(N, device=DEV), _ws(1 << 20)
    for a, e in (((x.float(), w, b, None, y), TypeError), ((x, w.half(), b, None, y), TypeError), ((x, w.cpu(), b, None, y), TypeError),
                 ((x, w, b.half(), None, y), TypeError), ((x, w, b[:8], None, y), TypeError), ((x, w, b, g[:8], y), ValueError),
                 ((x, w, b, None, y[:, :32]), ValueError), ((x, w[:, :32], b, None, y), ValueError), ((x, w.t(), b, None, y), ValueError),
                 ((x[0], w, b, None, y), TypeError), ((x, w, b, None, y, g[:, :8]), ValueError),
                 ((x, w, b, None, y, None, "swish"), ValueError), ((x[:, :60], w[:, :60], b, None, y), rn.RmsNormError)):
        with pytest.raises(e):
            rn.linear_fwd(*a)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for a, e in (((g, x, w, None, dx, dw, b, ws, "gelu"), TypeError), ((g, x, w, None, dw, dw, b, ws), ValueError),
                 ((g, x, w, None, dx, dx, b, ws), ValueError), ((g, x, w, None, dx, dw, b.double(), ws), TypeError),
                 ((g, x, w, None, dx, dw, b, ws[:16]), rn.RmsNormError), ((g, x, w, None, dx, dw, b, ws.cpu()), TypeError)):
        with pytest.raises(e):
            rn.linear_bwd(*a)
    for a, e in (((x, w, w[:8], y), ValueError), ((x, w, w, y, y, None), TypeError), ((x, w, w, y, None, None, "none "), ValueError)):
        with pytest.raises(e):
            rn.linear_gated_fwd(*a)
    for a, e in (((g, x, w, w, g, g, dx, dw, None, ws), TypeError), ((g, x, w, w, g, None, dx, dw, dw, ws), (TypeError, AttributeError)),
                 ((g, x, w, w, g, g, dx, dw, dw, ws[:16]), rn.RmsNormError)):
        with pytest.raises(e):
            rn.linear_gated_bwd(*a)
