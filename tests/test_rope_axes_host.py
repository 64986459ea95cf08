"""Host checks (no GPU) of rotary positions of several axes: refusals before any
launch, the pairs' axes, and the 64-bit definitions of the GPU tests against differences."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import build as cuda_build
from tests import axes_ref as ref
from tests.test_block_host import A, EALIGN, EINVAL, EWORKSPACE, ROPE_BAD, _differences, _Slots


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return rn.load()


def _turn(lib, fn="rope_axes_fwd", q=A, qs=(256, 64), k=A, ks=(128, 64), f=A, ax=A, n=3, pos=A, ps=(4, 1), p64=1, qo=2 * A,
          qos=(256, 64), ko=2 * A, kos=(128, 64), T=4, Hq=4, Hk=2, D=64, R=64, scale=1.0, layout=0, dtype=0):
    return getattr(lib, fn)(q, *qs, k, *ks, f, ax, n, pos, *ps, p64, qo, *qos, ko, *kos, T, Hq, Hk, D, R, scale, layout, dtype,
                            None)


def _norm_fwd(lib, w=A, r=A, eps=1e-6, q=A, qs=(256, 64), k=A, ks=(128, 64), f=A, ax=A, n=3, pos=A, ps=(4, 1), p64=1, qo=2 * A,
              qos=(256, 64), ko=2 * A, kos=(128, 64), T=4, Hq=4, Hk=2, D=64, R=64, scale=1.0, layout=0, dtype=0):
    return lib.rmsnorm_rope_axes_fwd(q, *qs, k, *ks, w, A, f, ax, n, pos, *ps, p64, qo, *qos, ko, *kos, r, A, T, Hq, Hk, D, R,
                                     scale, layout, eps, 0, dtype, None)


def _norm_bwd(lib, w=A, r=A, x=A, dw=A, ws=A, size=1 << 40, q=A, qs=(256, 64), k=A, ks=(128, 64), f=A, ax=A, n=3, pos=A,
              ps=(4, 1), p64=1, qo=2 * A, qos=(256, 64), ko=2 * A, kos=(128, 64), T=4, Hq=4, Hk=2, D=64, R=64, scale=1.0, layout=0,
              dtype=0):
    return lib.rmsnorm_rope_axes_bwd(q, *qs, k, *ks, x, 256, 64, A, 128, 64, w, A, f, ax, n, pos, *ps, p64, r, A, qo, *qos, ko,
                                     *kos, dw, A, ws, size, T, Hq, Hk, D, R, scale, layout, 0, dtype, None)


BAD = ROPE_BAD + [(dict(ax=0), EINVAL), (dict(pos=0), EINVAL), (dict(n=0), EINVAL), (dict(n=-1), EINVAL), (dict(n=257), EINVAL),
                  (dict(ps=(-4, 1)), EINVAL), (dict(ps=(4, -1)), EINVAL), (dict(ps=(1 << 62, 1)), EINVAL),
                  (dict(ps=(4, 1 << 62)), EINVAL)]


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("bad,status", BAD)
def test_refusals(lib, bad, status, slots):
    by = _Slots(lib) if slots else lib
    for fn in ("rope_axes_fwd", "rope_axes_bwd"):
        assert _turn(by, fn, **bad) == status
    assert _norm_fwd(by, **bad) == status and _norm_bwd(by, **bad) == status


@pytest.mark.parametrize("slots", [False, True])
def test_refusals_of_the_norm(lib, slots):
    by = _Slots(lib) if slots else lib
    for bad, status in ((dict(w=0), EINVAL), (dict(w=A + 4), EALIGN), (dict(r=0), EINVAL)):
        assert _norm_fwd(by, **bad) == _norm_bwd(by, **bad) == status
    assert _norm_fwd(by, eps=-1.0) == EINVAL
    for bad, status in ((dict(x=0), EINVAL), (dict(dw=0), EINVAL), (dict(ws=0), EWORKSPACE), (dict(size=16), EWORKSPACE),
                        (dict(ws=A + 8), EALIGN)):
        assert _norm_bwd(by, **bad) == status
    for fn in (_turn, _norm_fwd):
        assert fn(by, T=0, q=0, k=0, qo=0, ko=0, f=0, ax=0, pos=0) == 0


# --------------------------------------------------------------------------
# the pairs' axes
# --------------------------------------------------------------------------
def test_axes_side_by_side():
    assert rn.rope_axes_map((2, 3, 1)).tolist() == [0, 0, 1, 1, 1, 2]
    assert rn.rope_axes_map((4,)).tolist() == [0] * 4
    assert rn.rope_axes_map((128, 64, 64)).numel() == 256


def test_axes_dealt_in_turn():
    assert rn.rope_axes_map((4, 2, 2), True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert rn.rope_axes_map((2, 2), True).tolist() == [0, 1, 0, 1]
    assert rn.rope_axes_map((3, 1), True).tolist() == [0, 1, 0, 0]
    for s in ((24, 20, 20), (16, 8, 8), (5, 4, 3, 2)):
        m = rn.rope_axes_map(s, True).tolist()
        assert [m.count(a) for a in range(len(s))] == list(s)
        assert all(m[i] == i % len(s) for i in range(len(s) * min(s)))


@pytest.mark.parametrize("sections,cycled", [((), False), ((0, 4), False), ((4, -1), False), ((200, 57), False), ((1, 3), True),
                                             ((2, 3, 3), True), ((300,), False)])
def test_axes_refused(sections, cycled):
    with pytest.raises(rn.RmsNormError, match="EINVAL"):
        rn.rope_axes_map(sections, cycled)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        rn.rope_axes_fwd(x, None, torch.zeros(32, dtype=torch.float64), torch.zeros(32, dtype=torch.uint8), x, None,
                         torch.zeros((2, 2), dtype=torch.int64))


# --------------------------------------------------------------------------
# the 64-bit definitions
# --------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    gen = torch.Generator().manual_seed(4)
    x, g, w = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((2, 3, 16), (2, 3, 16), (16,)))
    pos, f, axis = torch.tensor([[5, 700], [3, 9], [1, 0]]), rn.rope_frequencies(12), rn.rope_axes_map((2, 2, 2), True)
    turn = lambda: (ref.turned(x, pos, axis, f, 1.5, interleaved)[0] * g).sum()
    torch.testing.assert_close(ref.turned(g, pos, axis, f, 1.5, interleaved, back=True)[0], _differences(turn, x), rtol=1e-7,
                               atol=1e-8)
    fused = lambda: (ref.norm_turn_fwd(x, w, 1e-6, pos, axis, f, 1.5, interleaved)[0][0] * g).sum()
    rstd = ref.norm_turn_fwd(x, w, 1e-6, pos, axis, f, 1.5, interleaved)[0][1]
    dx, dw = ref.norm_turn_bwd(g, x, w, rstd, pos, axis, f, 1.5, interleaved)[0]
    torch.testing.assert_close(dx, _differences(fused, x), rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(dw, _differences(fused, w), rtol=1e-7, atol=1e-8)


def test_equal_positions_are_one_axis():
    from tests import block_ref

    gen = torch.Generator().manual_seed(6)
    x = torch.randn((4, 2, 16), generator=gen, dtype=torch.float64)
    p, f = torch.tensor([0, 1, -7, 100000]), rn.rope_frequencies(16)
    a = ref.turned(x, p.expand(3, 4), rn.rope_axes_map((4, 2, 2)), f, 1.25, True)
    b = block_ref.turned(x, p, f, 1.25, True)
    torch.testing.assert_close(a[0], b[0], rtol=1e-9, atol=1e-9)
    torch.testing.assert_close(a[1], b[1], rtol=1e-12, atol=0)
