"""Projections and gated blocks of the same values in other layouts: rows that start on
lines of 128 bytes and rows that do not take tiles of other sizes, and have the same bits."""
from __future__ import annotations

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import synth
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
# (T, K, N), together with every change of rows a CTA, of 128 to 256 columns and between single CTAs and pairs that the
# tiles' model makes for rows that do not start on lines, forward, gated, and of both gradients
SIZES = [(3000, 2056, 1032), (300, 2056, 4104), (129, 264, 1024), (200, 4096, 2000), (129, 264, 4104), (2048, 264, 1024),
         (129, 4096, 2000), (129, 4096, 4104), (1021, 4096, 520), (1021, 4096, 1024)]


def _laid(t, extra, first):
    """t's values in rows a multiple of 64 and ``extra`` apart, from the ``first`` value of a line on."""
    rows, cols = t.shape
    ld = -(-cols // 64) * 64 + extra
    base = torch.full((rows * ld + 64,), float("nan"), dtype=t.dtype, device=DEV)
    v = base[first:first + rows * ld].view(rows, ld)[:, :cols]
    return v.copy_(t)


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,act", [(BF16, "silu"), (F16, "gelu_tanh")])
def test_bits_do_not_depend_on_the_layout(T, K, N, dtype, act):
    def mat(r, c, seed, std=1.0):
        return (synth.normal16((r, c), seed, DEV, dtype=F16).float() * std).to(dtype)

    x, g, r, z, u = mat(T, K, 1), mat(T, N, 2, 0.25), mat(T, N, 3), mat(T, N, 4), mat(T, N, 5)
    w, v, b = mat(N, K, 6, K ** -0.5), mat(N, K, 7, K ** -0.5), synth.gamma_f32(N, 8, DEV)
    ws = torch.full((max(rn.linear_bwd_workspace_bytes(T, N, K, act), rn.linear_gated_bwd_workspace_bytes(T, N, K)),), 255,
                    dtype=torch.uint8, device=DEV)

    def step(extra, first):
        at = lambda t: _laid(t, extra, first)
        out = lambda like: at(torch.zeros_like(like))
        X, G, R, Z, U, W, V = (at(t) for t in (x, g, r, z, u, w, v))
        y, zz, h, gate, up = (out(g) for _ in range(5))
        rn.linear_fwd(X, W, b, R, y, zz, act)
        rn.linear_gated_fwd(X, W, V, h, gate, up, act)
        dx, dw, db, dx0, dw0 = out(x), out(w), torch.empty(N, device=DEV), out(x), out(w)
        rn.linear_bwd(G, X, W, Z, dx, dw, db, ws, act)
        rn.linear_bwd(G, X, W, None, dx0, dw0, None, ws)
        dh, dwg, dwu = out(x), out(w), out(w)
        rn.linear_gated_bwd(G, X, W, V, Z, U, dh, dwg, dwu, ws, act)
        return [t.contiguous() for t in (y, zz, h, gate, up, dx, dw, db, dx0, dw0, dh, dwg, dwu)]

    lines = step(0, 0)
    for extra, first in ((8, 0), (0, 8), (24, 40)):
        for i, (p, q) in enumerate(zip(lines, step(extra, first))):
            assert torch.equal(p, q), (i, extra, first)
