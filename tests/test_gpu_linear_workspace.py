"""Workspaces of the projections' gradients on the GPU: a call asks for what its outputs
take, writes nothing beyond it, and has the same bits as one with every output."""
from __future__ import annotations

import itertools

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _mat(rows, cols, seed, std=1.0):
    return (synth.normal16((rows, cols), seed, DEV, dtype=torch.float16).float() * std).to(BF16)


def _pad(n):
    return -(-n // 256) * 256


def _db_rows(T, N):
    """Bytes of db's partial rows: ranges of 32 rows and more, 1824 over the columns' groups of 256."""
    return _pad(4 * N * max(1, min(-(-1824 // -(-N // 256)), -(-T // 32))))


def _guarded(n):
    """n bytes of NaN between guards."""
    base = torch.full((n + 512,), 255, dtype=torch.uint8, device=DEV)
    base[:256], base[256 + n:] = 77, 77
    return base, base[256:256 + n]


def _intact(base, n):
    assert bool((base[:256] == 77).all()) and bool((base[256 + n:] == 77).all())


@pytest.mark.parametrize("T,K,N", [(9000, 264, 136), (300, 264, 520), (1, 64, 40)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_bwd_asks_for_what_its_outputs_take(T, K, N, act):
    x, g, w, z = _mat(T, K, 1), _mat(T, N, 2), _mat(N, K, 3), _mat(T, N, 4)
    new = lambda: [torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)]
    full = new()
    every = rn.linear_bwd_workspace_bytes(T, N, K, act)
    rn.linear_bwd(g, x, w, z, *full, torch.empty(every, dtype=torch.uint8, device=DEV), act)
    dz = 0 if act == "none" else _pad(2 * T * N)
    sums = every - dz - _db_rows(T, N)
    assert (sums > 0) == (T == 9000)
    for wanted in itertools.product((False, True), repeat=3):
        need = (dz if wanted[0] or wanted[1] else 0) + (sums if wanted[1] else 0) + (_db_rows(T, N) if wanted[2] else 0)
        out = [t if on else None for t, on in zip(new(), wanted)]
        base, ws = _guarded(need)
        rn.linear_bwd(g, x, w, z, *out, ws if need else None, act)
        _intact(base, need)
        assert all(b is None or torch.equal(a, b) for a, b in zip(full, out)), wanted
        if need:
            for short in (None, ws[:need - 1]):
                with pytest.raises(rn.RmsNormError, match="EWORKSPACE"):
                    rn.linear_bwd(g, x, w, z, *out, short, act)


@pytest.mark.parametrize("T,K,N", [(18432, 520, 1032), (300, 264, 520), (1, 64, 40)])
def test_linear_gated_bwd_asks_for_what_its_outputs_take(T, K, N):
    x, g, wg, wu, gate, up = _mat(T, K, 1), _mat(T, N, 2), _mat(N, K, 3), _mat(N, K, 4), _mat(T, N, 5), _mat(T, N, 6)
    full = [torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)]
    every = rn.linear_gated_bwd_workspace_bytes(T, N, K)
    rn.linear_gated_bwd(g, x, wg, wu, gate, up, *full, torch.empty(every, dtype=torch.uint8, device=DEV))
    for dx, dw, need in ((True, False, 2 * _pad(2 * T * N)), (False, True, every), (False, False, 0)):
        out = [torch.empty_like(t) if on else None for t, on in zip(full, (dx, dw, dw))]
        base, ws = _guarded(need)
        rn.linear_gated_bwd(g, x, wg, wu, gate, up, *out, ws if need else None)
        _intact(base, need)
        assert all(b is None or torch.equal(a, b) for a, b in zip(full, out))
        if need:
            for short in (None, ws[:need - 1]):
                with pytest.raises(rn.RmsNormError, match="EWORKSPACE"):
                    rn.linear_gated_bwd(g, x, wg, wu, gate, up, *out, short)


def test_one_workspace_for_every_number_of_rows():
    """The size of the largest T alone would be refused at a smaller one."""
    K, N, T_max = 520, 1032, 18433
    ws = torch.empty(rn.linear_gated_bwd_workspace_bytes_max(T_max, N, K), dtype=torch.uint8, device=DEV)
    assert rn.linear_gated_bwd_workspace_bytes(18432, N, K) > rn.linear_gated_bwd_workspace_bytes(T_max, N, K)
    x, g, wg, wu, gate, up = _mat(T_max, K, 1), _mat(T_max, N, 2), _mat(N, K, 3), _mat(N, K, 4), _mat(T_max, N, 5), _mat(T_max, N, 6)
    for T in (T_max, 18432, 9000, 70, 1):
        a, b = ([torch.empty_like(x[:T]), torch.empty_like(wg), torch.empty_like(wu)] for _ in range(2))
        args = (g[:T], x[:T], wg, wu, gate[:T], up[:T])
        rn.linear_gated_bwd(*args, *a, ws)
        rn.linear_gated_bwd(*args, *b, torch.empty(rn.linear_gated_bwd_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
