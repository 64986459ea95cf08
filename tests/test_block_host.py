"""Host checks (no GPU) of LayerNorm, rotary positions and the head RMSNorm with
rotary positions: exports and prototypes, refusals before any launch, the
frequencies, and the 64-bit definitions of the GPU tests against differences."""
from __future__ import annotations

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import build as cuda_build
from tests import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an address that is never followed

EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return rn.load()


def _declared(header):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return [(r.split()[-1], n, [p.strip() for p in args.split(",")])
            for r, n, args in re.findall(r"\b((?:int|size_t))\s+((?:layernorm|rope|rmsnorm_rope)_\w+)\s*\(([^)]*)\)", txt)]


_TYPES = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "double": ctypes.c_double,
          "size_t": ctypes.c_size_t, "rmsn_stream": ctypes.c_void_p}


@pytest.mark.parametrize("header,names", [("layernorm.h", "LAYERNORM_SYMBOLS"), ("rope.h", "ROPE_SYMBOLS"),
                                          ("rmsnorm.h", None)])
def test_prototypes_match_the_headers(lib, header, names):
    decls = _declared(header)
    want = set(getattr(rn, names)) if names else {n for n in rn.EXPORTED_SYMBOLS if n.startswith("rmsnorm_rope")}
    assert {n for _, n, _ in decls} == want and want
    for ret, name, params in decls:
        res, args = rn._SIGS[name]
        assert hasattr(lib, name) and res is _TYPES[ret] and len(args) == len(params), name
        for p, ct in zip(params, args):
            assert ct is (ctypes.c_void_p if "*" in p else _TYPES[p.split()[0]]), (name, p)


def test_a_c_program_links_every_entry_point(lib, tmp_path):
    names = [*rn.LAYERNORM_SYMBOLS, *rn.ROPE_SYMBOLS, *rn.SLOTS_SYMBOLS]
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text('#include <stdio.h>\n#include "layernorm.h"\n#include "rope.h"\n#include "slots.h"\ntypedef void (*fn)(void);\n'
                   "static const fn all[] = {" + ", ".join(f"(fn){n}" for n in names) + "};\n"
                   "int main(void) {\n  double f[4];\n"
                   "  const int st = rope_frequencies(8, 10000.0, ROPE_SCALING_NONE, 1.0, 0, 0, 0, f);\n"
                   '  printf("%zu %zu %d %.17g\\n", sizeof all / sizeof all[0], layernorm_bwd_workspace_bytes(100, 64),'
                   " st, f[1]);\n  return 0;\n}\n")
    so = cuda_build.lib_path()
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe), "-L", os.path.dirname(so), "-l:" + os.path.basename(so),
                    "-Wl,-rpath," + os.path.dirname(so)], check=True)
    n, ws, st, f1 = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert int(n) == len(names) and int(ws) == rn.layernorm_bwd_workspace_bytes(100, 64)
    assert int(st) == 0 and float(f1) == pytest.approx(0.1, rel=1e-15)


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def _ln_fwd(lib, x=A, ldx=64, w=A, b=A, y=A, ldy=64, m=A, r=A, T=4, D=64, eps=1e-5, dtype=0):
    return lib.layernorm_fwd(x, ldx, w, b, y, ldy, m, r, T, D, eps, 0, dtype, None)


def _ln_bwd(lib, g=A, x=A, w=A, m=A, r=A, dx=A, ld=64, dw=A, db=A, ws=A, size=1 << 40, T=4, D=64, dtype=0):
    return lib.layernorm_bwd(g, ld, x, ld, w, m, r, dx, ld, dw, db, ws, size, T, D, 0, dtype, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), EINVAL), (dict(D=60), EUNSUPPORTED), (dict(D=16392, ldx=16392, ldy=16392), EUNSUPPORTED),
    (dict(D=0), EUNSUPPORTED), (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(x=0), EINVAL),
    (dict(x=A + 2), EALIGN), (dict(ldx=68), EALIGN), (dict(ldx=56), EINVAL), (dict(y=0), EINVAL),
    (dict(w=0), EINVAL), (dict(w=A + 4), EALIGN), (dict(b=A + 4), EALIGN), (dict(m=0), EINVAL), (dict(r=A + 8), EALIGN),
    (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=math.inf), EINVAL)])
def test_layernorm_fwd_refuses(lib, bad, status):
    assert _ln_fwd(lib, **bad) == status
    assert _ln_fwd(lib, T=0, x=0, y=0, w=0, b=0, m=0, r=0) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=-1), EINVAL), (dict(D=12), EUNSUPPORTED), (dict(g=0), EINVAL), (dict(x=A + 8), EALIGN),
    (dict(dx=0), EINVAL), (dict(ld=60), EINVAL), (dict(ld=70), EALIGN), (dict(dw=0), EINVAL), (dict(dw=0, T=0), EINVAL),
    (dict(db=A + 4), EALIGN), (dict(w=0), EINVAL), (dict(m=0), EINVAL), (dict(r=0), EINVAL), (dict(ws=0), EWORKSPACE),
    (dict(size=16), EWORKSPACE), (dict(ws=A + 4), EALIGN)])
def test_layernorm_bwd_refuses(lib, bad, status):
    assert _ln_bwd(lib, **bad) == status


def _rope(lib, fn="rope_fwd", q=A, qs=(256, 64), k=A, ks=(128, 64), f=A, pos=A, p64=1, qo=2 * A, qos=(256, 64), ko=2 * A,
          kos=(128, 64), T=4, Hq=4, Hk=2, D=64, R=64, scale=1.0, layout=0, dtype=0):
    return getattr(lib, fn)(q, *qs, k, *ks, f, pos, p64, qo, *qos, ko, *kos, T, Hq, Hk, D, R, scale, layout, dtype, None)


ROPE_BAD = [
    (dict(dtype=3), EINVAL), (dict(layout=2), EINVAL), (dict(p64=2), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(scale=math.inf), EINVAL), (dict(D=60), EUNSUPPORTED), (dict(D=520, R=64), EUNSUPPORTED),
    (dict(R=0), EUNSUPPORTED), (dict(R=63), EUNSUPPORTED), (dict(R=66), EUNSUPPORTED), (dict(R=-2), EUNSUPPORTED),
    (dict(Hq=0), EINVAL), (dict(Hk=-1), EINVAL), (dict(Hq=65537), EINVAL), (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL),
    (dict(q=0), EINVAL), (dict(k=0), EINVAL), (dict(q=A + 2), EALIGN), (dict(qs=(260, 64)), EALIGN),
    (dict(ks=(128, 68)), EALIGN), (dict(qs=(-256, 64)), EINVAL), (dict(qs=(1 << 62, 64)), EINVAL), (dict(f=0), EINVAL),
    (dict(f=A + 8), EALIGN), (dict(pos=A + 4), EALIGN), (dict(qo=0), EINVAL), (dict(ko=2 * A + 8), EALIGN),
    (dict(qos=(248, 64)), EINVAL), (dict(qos=(64, 64)), EINVAL), (dict(qos=(256, 0)), EINVAL),
    (dict(kos=(0, 64)), EINVAL), (dict(qos=(64, 248)), EINVAL),
    (dict(qo=A, qos=(512, 64)), EINVAL), (dict(ko=A, ks=(64, 256)), EINVAL)]  # in place with other strides


@pytest.mark.parametrize("fn", ["rope_fwd", "rope_bwd"])
@pytest.mark.parametrize("bad,status", ROPE_BAD)
def test_rope_refuses(lib, fn, bad, status):
    assert _rope(lib, fn, **bad) == status
    assert _rope(lib, fn, T=0, q=0, k=0, qo=0, ko=0, f=0, pos=0) == 0


def _norm_fwd(lib, w=A, wk=A, r=A, rk=A, eps=1e-6, q=A, qs=(256, 64), k=A, ks=(128, 64), f=A, pos=A, p64=1, qo=2 * A,
              qos=(256, 64), ko=2 * A, kos=(128, 64), T=4, Hq=4, Hk=2, D=64, R=64, scale=1.0, layout=0, dtype=0):
    return lib.rmsnorm_rope_fwd(q, *qs, k, *ks, w, wk, f, pos, p64, qo, *qos, ko, *kos, r, rk, T, Hq, Hk, D, R, scale,
                                layout, eps, 0, dtype, None)


@pytest.mark.parametrize("bad,status", ROPE_BAD + [
    (dict(w=0), EINVAL), (dict(wk=0), EINVAL), (dict(w=A + 4), EALIGN), (dict(r=0), EINVAL), (dict(rk=A + 4), EALIGN),
    (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL)])
def test_norm_rope_fwd_refuses(lib, bad, status):
    assert _norm_fwd(lib, **bad) == status
    assert _norm_fwd(lib, T=0, q=0, k=0, qo=0, ko=0, f=0, pos=0, w=0, wk=0, r=0, rk=0) == 0


def _norm_bwd(lib, w=A, wk=A, r=A, rk=A, x=A, xs=(256, 64), xk=A, dw=A, dwk=A, ws=A, size=1 << 40, q=A, qs=(256, 64),
              k=A, ks=(128, 64), f=A, pos=A, p64=1, qo=2 * A, qos=(256, 64), ko=2 * A, kos=(128, 64), T=4, Hq=4, Hk=2,
              D=64, R=64, scale=1.0, layout=0, dtype=0):
    return lib.rmsnorm_rope_bwd(q, *qs, k, *ks, x, *xs, xk, *ks, w, wk, f, pos, p64, r, rk, qo, *qos, ko, *kos, dw, dwk,
                                ws, size, T, Hq, Hk, D, R, scale, layout, 0, dtype, None)


@pytest.mark.parametrize("bad,status", ROPE_BAD + [
    (dict(w=0), EINVAL), (dict(wk=0), EINVAL), (dict(r=0), EINVAL), (dict(rk=A + 4), EALIGN), (dict(x=0), EINVAL),
    (dict(xk=A + 2), EALIGN), (dict(xs=(260, 64)), EALIGN), (dict(dw=0), EINVAL), (dict(dwk=A + 4), EALIGN),
    (dict(dw=0, T=0), EINVAL), (dict(ws=0), EWORKSPACE), (dict(size=16), EWORKSPACE), (dict(ws=A + 8), EALIGN)])
def test_norm_rope_bwd_refuses(lib, bad, status):
    assert _norm_bwd(lib, **bad) == status


class _Slots:
    """The library through ``norm_call``."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        entry, pack, n = rn._SLOTS[name]
        return lambda *args: self.lib.norm_call(entry, pack(*(0 if a is None else a for a in args)), n)


@pytest.mark.parametrize("bad,status", ROPE_BAD + [(dict(w=0), EINVAL), (dict(wk=A + 4), EALIGN), (dict(r=0), EINVAL),
                                                   (dict(dtype=7), EINVAL), (dict(T=0), 0)])
def test_arguments_in_an_array_are_the_same_arguments(lib, bad, status):
    """Every refusal depends on the argument at its own place, so the array's order is the prototype's."""
    by_array = _Slots(lib)
    if not {"w", "wk", "r"} & set(bad):
        for fn in ("rope_fwd", "rope_bwd"):
            assert _rope(by_array, fn, **bad) == _rope(lib, fn, **bad) == status
    assert _norm_fwd(by_array, **bad) == _norm_fwd(lib, **bad) == status
    if bad != dict(T=0):
        assert _norm_bwd(by_array, **bad) == _norm_bwd(lib, **bad) == status
    ln = {k: v for k, v in bad.items() if k in ("w", "r", "dtype", "T")}
    if ln == bad:
        assert _ln_fwd(by_array, **bad) == _ln_fwd(lib, **bad) == status
        if bad != dict(T=0):
            assert _ln_bwd(by_array, **bad) == _ln_bwd(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [(dict(eps=-1.0), EINVAL), (dict(eps=1e300), EINVAL), (dict(eps=math.nan), EINVAL)])
def test_floats_in_an_array(lib, bad, status):
    assert _ln_fwd(_Slots(lib), **bad) == _norm_fwd(_Slots(lib), **bad) == status


def test_arrays_that_are_not_the_entry_points(lib):
    for name, (entry, pack, n) in rn._SLOTS.items():
        assert n == len(rn._SIGS[name][1])
        good = pack(*[0] * n)
        assert lib.norm_call(entry, good, n - 1) == lib.norm_call(entry, good, n + 1) == EINVAL
        assert lib.norm_call(entry, None, n) == EINVAL
    assert lib.norm_call(len(rn._SLOTS), good, n) == lib.norm_call(-1, good, n) == EINVAL
    assert _rope(_Slots(lib), layout=1 << 32) == EINVAL and _rope(_Slots(lib), dtype=(1 << 32) + 1) == EINVAL
    enum = re.findall(r"NORM_(\w+)\s*=\s*(\d+)", open(os.path.join(ROOT, "include", "slots.h")).read())
    assert {n.lower(): int(v) for n, v in enum} == {n: e for n, (e, _, _) in rn._SLOTS.items()}


def test_workspace_queries(lib):
    assert rn.layernorm_bwd_workspace_bytes(0, 64) == 0 and rn.layernorm_bwd_workspace_bytes(5, 60) == 0
    assert rn.layernorm_bwd_workspace_bytes(1, 64) == 2 * 64 * 4
    assert rn.rmsnorm_rope_bwd_workspace_bytes(0, 4, 2, 64) == 0 and rn.rmsnorm_rope_bwd_workspace_bytes(5, 0, 2, 64) == 0
    assert rn.rmsnorm_rope_bwd_workspace_bytes(5, 4, 2, 520) == 0
    for D in (8, 128, 256, 264, 1000, 4096, 8200, 16384):
        for T_max in (1, 7, 300, 305, 4000, 40000):
            most = max(rn.layernorm_bwd_workspace_bytes(t, D) for t in range(1, T_max + 1))
            assert most <= rn.layernorm_bwd_workspace_bytes_max(T_max, D) <= 1.1 * most + 8 * D, (T_max, D)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    v = torch.zeros(64)
    with pytest.raises(TypeError, match="CUDA"):
        rn.layernorm_fwd(x, v, None, x, v, v)
    with pytest.raises(TypeError, match="CUDA"):
        rn.rope_fwd(x.view(2, 1, 64), None, v.double(), x.view(2, 1, 64), None)


# --------------------------------------------------------------------------
# frequencies
# --------------------------------------------------------------------------
@pytest.mark.parametrize("R", [2, 8, 24, 64, 128, 512])
def test_frequencies(lib, R):
    i = torch.arange(R // 2, dtype=torch.float64)
    plain = rn.rope_frequencies(R, 10000.0)
    want = torch.tensor([math.exp(-math.log(10000.0) * 2 * k / R) for k in range(R // 2)], dtype=torch.float64)
    torch.testing.assert_close(plain, want, rtol=1e-13, atol=0)
    torch.testing.assert_close(rn.rope_frequencies(R, scaling="linear", factor=4.0), want / 4, rtol=1e-13, atol=0)
    if R > 2:
        based = rn.rope_frequencies(R, scaling="base", factor=4.0)
        assert based[0] == 1.0
        torch.testing.assert_close(based[-1], want[-1] / 4, rtol=1e-12, atol=0)  # the slowest pair is interpolated
    turns = 4096.0 * want / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0, 1)
    torch.testing.assert_close(rn.rope_frequencies(R, scaling="ramp_turns", factor=8.0, low=1.0, high=32.0, length=4096.0),
                               want * (keep + (1 - keep) / 8), rtol=1e-13, atol=0)
    ramp = rn.rope_frequencies(R, scaling="ramp_index", factor=8.0, low=1.0, high=32.0, length=4096.0) / want
    assert bool((ramp <= 1 + 1e-12).all()) and bool((ramp >= 0.125 - 1e-12).all())
    assert bool((ramp[1:] <= ramp[:-1] + 1e-12).all())          # faster pairs keep more
    kept, interpolated = turns > 32.0 * 10000.0 ** (2 / R), turns < 10000.0 ** (-2 / R)  # a pair's step beyond the ramp
    torch.testing.assert_close(ramp[kept], torch.ones_like(ramp[kept]), rtol=1e-12, atol=0)
    torch.testing.assert_close(ramp[interpolated], torch.full_like(ramp[interpolated], 0.125), rtol=1e-12, atol=0)
    assert len(i) == len(plain)


@pytest.mark.parametrize("R,theta,length", [(64, 1e4, 65536.0), (64, 1e4, 4096.0), (128, 1e4, 131072.0), (128, 1e6, 32768.0),
                                            (32, 500.0, 1e7), (64, 1e4, 100.0), (8, 1e4, 3.0), (2, 1e4, 4096.0), (64, 1e4, 1e-30)])
@pytest.mark.parametrize("low,high", [(1.0, 32.0), (0.25, 4.0), (1.0, 1e300)])
def test_ramp_by_index_has_the_slope_of_its_definition(lib, R, theta, length, low, high):
    """From the pair that turns `high` times over `length` positions to the one that turns `low` times, whether or not
    the head has these pairs."""
    def index(turns):  # theta^(-2 i / R) length / 2 pi = turns
        return R * (math.log(length) - math.log(2 * math.pi * turns)) / (2 * math.log(theta))

    first, last = math.floor(index(high)), math.ceil(index(low))
    want = []
    for i in range(R // 2):
        k = min(1.0, max(0.0, (last - i) / (last - first)))
        want.append(math.exp(-math.log(theta) * 2 * i / R) * (k + (1 - k) / 16.0))
    got = rn.rope_frequencies(R, theta, "ramp_index", factor=16.0, low=low, high=high, length=length)
    # pow and exp(log) differ by a few of their arguments' roundings: |log f| 2^-53 and less
    torch.testing.assert_close(got, torch.tensor(want, dtype=torch.float64), rtol=1e-13, atol=0)


@pytest.mark.parametrize("kw", [dict(R=0), dict(R=3), dict(R=514), dict(theta=1.0), dict(theta=math.inf), dict(factor=0.5),
                                dict(factor=math.nan), dict(R=2, scaling="base", factor=2.0),
                                dict(scaling="ramp_turns", length=0.0), dict(scaling="ramp_turns", length=10.0, low=5.0, high=5.0),
                                dict(scaling="ramp_index", length=10.0, low=0.0)])
def test_frequencies_refuse(lib, kw):
    with pytest.raises(rn.RmsNormError, match="EINVAL"):
        rn.rope_frequencies(**{"R": 64, **kw})
    with pytest.raises(ValueError):
        rn.rope_frequencies(64, scaling="other")


# --------------------------------------------------------------------------
# the 64-bit definitions against differences
# --------------------------------------------------------------------------
def _differences(f, x, h=1e-5):
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        old = float(flat[i])
        flat[i] = old + h
        up = float(f())
        flat[i] = old - h
        o[i] = (up - float(f())) / (2 * h)
        flat[i] = old
    return out


def test_layernorm_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    x, g, w, b = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 16), (3, 16), (16,), (16,)))
    loss = lambda: (ref.ln_fwd(x, w, b, 1e-5)[0][0] * g).sum()
    _, mean, rstd = ref.ln_fwd(x, w, b, 1e-5)[0]
    for got, at in zip(ref.ln_bwd(g, x, w, mean, rstd)[0], (x, w, b)):
        torch.testing.assert_close(got, _differences(loss, at), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradients_against_differences(interleaved):
    gen = torch.Generator().manual_seed(4)
    x, g, w = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((2, 3, 16), (2, 3, 16), (16,)))
    pos, f = torch.tensor([5, 700]), rn.rope_frequencies(12)
    turn = lambda: (ref.turned(x, pos, f, 1.5, interleaved)[0] * g).sum()
    torch.testing.assert_close(ref.turned(g, pos, f, 1.5, interleaved, back=True)[0], _differences(turn, x), rtol=1e-7,
                               atol=1e-8)
    fused = lambda: (ref.norm_turn_fwd(x, w, 1e-6, pos, f, 1.5, interleaved)[0][0] * g).sum()
    rstd = ref.norm_turn_fwd(x, w, 1e-6, pos, f, 1.5, interleaved)[0][1]
    dx, dw = ref.norm_turn_bwd(g, x, w, rstd, pos, f, 1.5, interleaved)[0]
    torch.testing.assert_close(dx, _differences(fused, x), rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(dw, _differences(fused, w), rtol=1e-7, atol=1e-8)
