"""Gradients of the projections from saved fp16 values that overflowed: the forward
goes on with the fp32 value, so finite outputs may have an infinite z, gate or up behind them."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

F16 = torch.float16
ACTS = sorted(rn.LINEAR_ACTS)
INF = float("inf")
# act' at minus and plus infinity
LIMITS = {"none": (1.0, 1.0), "silu": (0.0, 1.0), "sigmoid": (0.0, 0.0), "gelu": (0.0, 1.0), "gelu_tanh": (0.0, 1.0),
          "relu": (0.0, 1.0)}


def _full(rows, cols, value=0.0):
    return torch.full((rows, cols), value, dtype=F16, device=DEV)


def _column(values):
    """[T, 8] with the values in every column."""
    return torch.tensor(values, device=DEV)[:, None].expand(len(values), 8).contiguous().to(F16)


def _ws(n):
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_slopes_of_an_overflowed_z(act):
    """z = +-90000 of finite fp16 inputs, saved as infinite: dz is g times the slope's limit."""
    T = 4
    x, w = _full(T, 8), _full(8, 8)
    x[:, 0], w[:, 0] = torch.tensor([300.0, -300.0, 1.0, -1.0], device=DEV), 300.0
    y, z = _full(T, 8), _full(T, 8)
    rn.linear_fwd(x, w, None, None, y, z, act)
    assert z[:2, 0].tolist() == [INF, -INF] and bool(y[1:].isfinite().all())
    g = _column([0.5, -2.0, 0.0, 0.0])
    dx, dw, db = _full(T, 8), _full(8, 8), torch.empty(8, device=DEV)
    rn.linear_bwd(g, x, w, z, dx, dw, db, _ws(rn.linear_bwd_workspace_bytes(T, 8, 8, act)), act)
    low, high = LIMITS[act]
    dz = torch.tensor([0.5 * high, -2.0 * low, 0.0, 0.0])  # exact, and so are the sums of eight
    assert torch.equal(dx[:, 0].cpu().float(), 8.0 * 300.0 * dz) and bool((dx[:, 1:] == 0).all())
    assert bool((dw[:, 0] == float((dz * x[:, 0].cpu().float()).sum())).all()) and bool((dw[:, 1:] == 0).all())
    assert bool((db == float(dz.sum())).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate,up,g", [(INF, 0.5, 0.0), (INF, 0.5, 2.0), (-INF, 0.5, 2.0), (-INF, INF, 2.0), (INF, INF, 0.0),
                                       (2.0, INF, 0.0), (-INF, 0.0, 2.0), (-INF, 0.0, 0.0)])
def test_gated_gradients_of_overflowed_values(act, gate, up, g):
    """One row, so that no infinity meets another row's zeros in the product: dwg and dwu are dgate and dup themselves."""
    x, w, dwg, dwu = _full(1, 8, 1.0), _full(8, 8), _full(8, 8), _full(8, 8)
    rn.linear_gated_bwd(_column([g]), x, w, w, _column([gate]), _column([up]), None, dwg, dwu,
                        _ws(rn.linear_gated_bwd_workspace_bytes(1, 8, 8)), act)
    low, high = LIMITS[act]
    slope = {INF: high, -INF: low}.get(gate, 1.0)
    value = {INF: 1.0 if act == "sigmoid" else INF, -INF: -INF if act == "none" else 0.0}.get(gate, 1.0)
    assert bool((dwg == (g * slope * up if g * slope * up == g * slope * up else 0.0)).all()), dwg
    assert bool((dwu == (g * value if g else 0.0)).all()), dwu


@pytest.mark.parametrize("act", ACTS)
def test_nan_stays(act):
    nan = float("nan")
    g, gate, up = _column([1.0, 1.0]), _column([nan, 1.0]), _column([1.0, nan])
    x, w, dwg, dwu = _full(2, 8, 1.0), _full(8, 8), _full(8, 8), _full(8, 8)
    rn.linear_gated_bwd(g[:1], x[:1], w, w, gate[:1], up[:1], None, dwg, dwu, _ws(rn.linear_gated_bwd_workspace_bytes(1, 8, 8)), act)
    assert bool(dwu.isnan().all()) and bool((dwg == 1.0).all() if act == "none" else dwg.isnan().all())
    rn.linear_gated_bwd(g[1:], x[1:], w, w, gate[1:], up[1:], None, dwg, dwu, _ws(rn.linear_gated_bwd_workspace_bytes(1, 8, 8)), act)
    assert bool(dwg.isnan().all()) and bool(dwu.isfinite().all())
    if act != "none":
        db = torch.empty(8, device=DEV)
        rn.linear_bwd(g, x, w, gate, None, None, db, _ws(rn.linear_bwd_workspace_bytes(2, 8, 8, act)), act)
        assert bool(db.isnan().all())
