"""Host checks (no GPU) of the projections' workspaces: one size for every T up to a
maximum, although the size of a T may fall as T grows, and what a call asks for."""
from __future__ import annotations

import random

import pytest

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import build as cuda_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return rn.load()


QUERIES = [(rn.linear_bwd_workspace_bytes, rn.linear_bwd_workspace_bytes_max, ("none",)),
           (rn.linear_bwd_workspace_bytes, rn.linear_bwd_workspace_bytes_max, ("gelu",)),
           (rn.linear_gated_bwd_workspace_bytes, rn.linear_gated_bwd_workspace_bytes_max, ())]


def _rows(T_max):
    """Every T at an end of its block of 64 rows or of a range's 512, up to T_max."""
    return sorted({t for b in range(64, T_max + 64, 64) for t in (b - 63, b - 1, b) if t <= T_max} | {T_max})


@pytest.mark.parametrize("N,K", [(4096, 4096), (6144, 4096), (1032, 520), (1024, 1024), (8, 8), (264, 136), (2056, 1000)])
@pytest.mark.parametrize("size,most,act", QUERIES)
def test_one_size_serves_every_smaller_T(N, K, size, most, act):
    T_max = 40000
    need = {t: size(t, N, K, *act) for t in _rows(T_max)}
    limits = [1, 64, 511, 512, 1023, 1024, 1025, 4097, 18432, 18433, 23680, 23681, 30000, 34816, 34817, 39999, 40000]
    for limit in limits:
        got, wanted = most(limit, N, K, *act), max(v for t, v in need.items() if t <= limit)
        # the activation's dz and db's rows are counted at T_max itself
        rest = got - wanted
        assert 0 <= rest <= 4 * limit * N + 512, (limit, got, wanted)
        assert got >= size(limit, N, K, *act)


def test_sizes_fall_as_rows_are_added():
    """The trap itself: a buffer of the larger T's size would be refused at the smaller."""
    for N, K, T in ((4096, 4096, 23680), (6144, 4096, 34816)):
        assert rn.linear_bwd_workspace_bytes(T, N, K) > 50 * rn.linear_bwd_workspace_bytes(T + 1, N, K)
        assert rn.linear_bwd_workspace_bytes_max(T + 1, N, K) == rn.linear_bwd_workspace_bytes(T, N, K)
    assert rn.linear_gated_bwd_workspace_bytes(18432, 1032, 520) > rn.linear_gated_bwd_workspace_bytes(18433, 1032, 520)


def test_at_any_sizes():
    rng = random.Random(3)
    log = lambda lo, hi: int(round(2.0 ** rng.uniform(lo, hi)))
    for _ in range(60):
        N, K = 8 * log(0, 12), 8 * log(0, 12)
        limit = log(9, 22)
        size, most, act = QUERIES[rng.randrange(3)]
        got = most(limit, N, K, *act)
        assert all(size(t, N, K, *act) <= got for t in {limit, *(rng.randint(1, limit) for _ in range(300))}), (limit, N, K)


def test_the_longest_axes_and_refusals():
    for N, K in ((8, 8), (1 << 20, 1 << 20), (4096, 4096), (8, 1 << 20)):
        T = (1 << 31) - 1
        assert rn.linear_bwd_workspace_bytes_max(T, N, K, "gelu") >= rn.linear_bwd_workspace_bytes(T, N, K, "gelu")
        assert rn.linear_gated_bwd_workspace_bytes_max(T, N, K) >= rn.linear_gated_bwd_workspace_bytes(T, N, K)
    for T, N, K in ((0, 64, 64), (-1, 64, 64), (1 << 31, 64, 64), (100, 60, 64), (100, 64, 60)):
        assert rn.linear_bwd_workspace_bytes_max(T, N, K) == rn.linear_gated_bwd_workspace_bytes_max(T, N, K) == 0
    with pytest.raises(ValueError):
        rn.linear_bwd_workspace_bytes_max(8, 8, 8, "swish")


# --------------------------------------------------------------------------
# what a call asks for (a workspace at an odd address: its size is looked at first, and nothing is launched)
# --------------------------------------------------------------------------
A = 1 << 20
EALIGN, EWORKSPACE = -2, -5


def _pad(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("T,N,K", [(4, 40, 64), (9000, 136, 264), (23680, 4096, 4096)])
@pytest.mark.parametrize("act", [0, 3])
@pytest.mark.parametrize("dx,dw,db", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (1, 1, 1)])
def test_linear_bwd_asks_for_what_its_outputs_take(lib, T, N, K, act, dx, dw, db):
    rows = _pad(4 * N * max(1, min(-(-1824 // -(-N // 256)), -(-T // 32))))
    dz = _pad(2 * T * N) if act else 0
    sums = rn.linear_bwd_workspace_bytes(T, N, K, "gelu" if act else "none") - dz - rows
    need = (dz if dx or dw else 0) + (rows if db else 0) + (sums if dw else 0)

    def call(ws, size):
        return lib.linear_bwd(A, N, A, K, A, K, A, N, A if dx else 0, K, A if dw else 0, K, A if db else 0, ws, size, T, N, K, act, 0,
                              None)

    if need:
        assert call(A + 8, need) == EALIGN and call(A + 8, need - 1) == call(0, need) == EWORKSPACE


def test_linear_gated_bwd_asks_for_no_sums_without_weights(lib):
    T, N, K = 18432, 1032, 520
    for dw, need in ((0, 2 * _pad(2 * T * N)), (A, rn.linear_gated_bwd_workspace_bytes(T, N, K))):
        def call(ws, size):
            return lib.linear_gated_bwd(A, N, A, K, A, K, A, K, A, N, A, N, A, K, dw, K, dw, K, ws, size, T, N, K, 1, 0, None)

        assert call(A + 8, need) == EALIGN and call(A + 8, need - 1) == call(0, need) == EWORKSPACE
