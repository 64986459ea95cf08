"""Host checks (no GPU) of the projections: exports and prototypes, refusals before
any launch, workspaces, and the 64-bit definitions of the GPU tests against differences."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

import invariant_rmsnorm_gb300 as rn
from invariant_rmsnorm_gb300 import build as cuda_build
from tests import linear_ref as ref
from tests.test_block_host import A, EALIGN, EINVAL, EUNSUPPORTED, EWORKSPACE, ROOT, _differences, _Slots

_TYPES = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "size_t": ctypes.c_size_t,
          "rmsn_stream": ctypes.c_void_p}


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return rn.load()


def test_prototypes_match_the_header(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "linear.h")).read(), flags=re.S)
    decls = re.findall(r"\b(int|size_t)\s+(linear_\w+)\s*\(([^)]*)\)", txt)
    assert {n for _, n, _ in decls} == set(rn.LINEAR_SYMBOLS)
    for ret, name, args in decls:
        params = [p.strip() for p in args.split(",")]
        res, sig = rn._SIGS[name]
        assert hasattr(lib, name) and res is _TYPES[ret] and len(sig) == len(params), name
        for p, ct in zip(params, sig):
            assert ct is (ctypes.c_void_p if "*" in p else _TYPES[p.split()[0]]), (name, p)
    acts = re.findall(r"LINEAR_ACT_(\w+)\s*=\s*(\d+)", txt)
    assert {n.lower(): int(v) for n, v in acts} == rn.LINEAR_ACTS


def test_a_c_program_links_every_entry_point(lib, tmp_path):
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text('#include <stdio.h>\n#include "linear.h"\ntypedef void (*fn)(void);\nstatic const fn all[] = {' +
                   ", ".join(f"(fn){n}" for n in rn.LINEAR_SYMBOLS) + "};\nint main(void) {\n"
                   '  printf("%zu %zu\\n", sizeof all / sizeof all[0], linear_bwd_workspace_bytes(100, 64, 32, LINEAR_ACT_GELU));\n'
                   "  return 0;\n}\n")
    so = cuda_build.lib_path()
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe), "-L", os.path.dirname(so), "-l:" + os.path.basename(so), "-Wl,-rpath," + os.path.dirname(so)],
                   check=True)
    n, ws = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert int(n) == len(rn.LINEAR_SYMBOLS) and int(ws) == rn.linear_bwd_workspace_bytes(100, 64, 32, "gelu")


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def _fwd(lib, x=A, ldx=64, w=A, ldw=64, b=A, r=2 * A, ldr=40, y=A, ldy=40, z=A, ldz=40, T=4, N=40, K=64, act=1, dtype=0):
    return lib.linear_fwd(x, ldx, w, ldw, b, r, ldr, y, ldy, z, ldz, T, N, K, act, dtype, None)


def _bwd(lib, g=A, ldg=40, x=A, ldx=64, w=A, ldw=64, z=A, ldz=40, dx=A, lddx=64, dw=A, lddw=64, db=A, ws=A, size=1 << 40, T=4,
         N=40, K=64, act=1, dtype=0):
    return lib.linear_bwd(g, ldg, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db, ws, size, T, N, K, act, dtype, None)


def _gated_fwd(lib, x=A, ldx=64, w=A, ldw=64, wu=A, ldwu=64, h=A, ldh=40, z=A, ldz=40, up=A, ldup=40, T=4, N=40, K=64, act=1,
               dtype=0):
    return lib.linear_gated_fwd(x, ldx, w, ldw, wu, ldwu, h, ldh, z, ldz, up, ldup, T, N, K, act, dtype, None)


def _gated_bwd(lib, g=A, ldg=40, x=A, ldx=64, w=A, ldw=64, wu=A, ldwu=64, z=A, ldz=40, up=A, ldup=40, dx=A, lddx=64, dw=A,
               lddw=64, dwu=A, lddwu=64, ws=A, size=1 << 40, T=4, N=40, K=64, act=1, dtype=0):
    return lib.linear_gated_bwd(g, ldg, x, ldx, w, ldw, wu, ldwu, z, ldz, up, ldup, dx, lddx, dw, lddw, dwu, lddwu, ws, size, T, N,
                                K, act, dtype, None)


ALL = [(dict(dtype=2), EINVAL), (dict(dtype=-1), EINVAL), (dict(act=-1), EINVAL), (dict(act=6), EINVAL), (dict(T=-1), EINVAL),
       (dict(T=1 << 31), EINVAL), (dict(N=36), EUNSUPPORTED), (dict(N=0), EUNSUPPORTED), (dict(K=60), EUNSUPPORTED),
       (dict(K=(1 << 20) + 8), EUNSUPPORTED), (dict(N=(1 << 20) + 8), EUNSUPPORTED), (dict(x=0), EINVAL), (dict(x=A + 2), EALIGN),
       (dict(ldx=56), EINVAL), (dict(ldx=68), EALIGN), (dict(ldx=(1 << 38) + 8), EINVAL), (dict(w=0), EINVAL),
       (dict(w=A + 8), EALIGN), (dict(ldw=68), EALIGN), (dict(ldw=56), EINVAL), (dict(ldz=36), EINVAL), (dict(z=A + 2), EALIGN)]
FORWARD = [(dict(T=0), 0), (dict(T=0, x=0, w=0), 0)]
BACKWARD = [(dict(g=0), EINVAL), (dict(g=A + 2), EALIGN), (dict(ldg=44), EALIGN), (dict(dx=A + 2), EALIGN), (dict(lddx=56), EINVAL),
            (dict(dw=A + 2), EALIGN), (dict(lddw=68), EALIGN), (dict(z=0), EINVAL), (dict(ws=0), EWORKSPACE),
            (dict(size=16), EWORKSPACE), (dict(ws=A + 8), EALIGN)]


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("bad,status", ALL + FORWARD + [
    (dict(y=0), EINVAL), (dict(y=A + 2), EALIGN), (dict(ldy=32), EINVAL), (dict(b=A + 4), EALIGN), (dict(r=2 * A + 2), EALIGN),
    (dict(ldr=44), EALIGN), (dict(r=A, ldr=48), EINVAL)])
def test_linear_fwd_refuses(lib, bad, status, slots):
    assert _fwd(_Slots(lib) if slots else lib, **bad) == status


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("bad,status", ALL + BACKWARD + [(dict(db=A + 4), EALIGN)])
def test_linear_bwd_refuses(lib, bad, status, slots):
    assert _bwd(_Slots(lib) if slots else lib, **bad) == status


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("bad,status", ALL + FORWARD + [
    (dict(wu=0), EINVAL), (dict(ldwu=68), EALIGN), (dict(h=0), EINVAL), (dict(ldh=32), EINVAL), (dict(z=0), EINVAL),
    (dict(up=0), EINVAL), (dict(up=A + 2), EALIGN), (dict(ldup=44), EALIGN)])
def test_gated_fwd_refuses(lib, bad, status, slots):
    assert _gated_fwd(_Slots(lib) if slots else lib, **bad) == status


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("bad,status", ALL + BACKWARD + [
    (dict(wu=0), EINVAL), (dict(up=0), EINVAL), (dict(ldup=44), EALIGN), (dict(dwu=0), EINVAL), (dict(lddwu=56), EINVAL),
    (dict(dw=0), EINVAL)])
def test_gated_bwd_refuses(lib, bad, status, slots):
    assert _gated_bwd(_Slots(lib) if slots else lib, **bad) == status


def test_workspaces(lib):
    assert rn.linear_bwd_workspace_bytes(0, 64, 64) == 0 and rn.linear_bwd_workspace_bytes(5, 60, 64) == 0
    assert rn.linear_gated_bwd_workspace_bytes(5, 64, 60) == 0
    for T, N, K in ((1, 8, 8), (1000, 264, 136), (9000, 264, 136), (8192, 4096, 4096)):
        none, gelu = (rn.linear_bwd_workspace_bytes(T, N, K, a) for a in ("none", "gelu"))
        assert none >= 4 * N and 2 * T * N <= gelu - none < 2 * T * N + 256
        assert rn.linear_gated_bwd_workspace_bytes(T, N, K) >= 4 * T * N
    with pytest.raises(ValueError):
        rn.linear_bwd_workspace_bytes(8, 8, 8, "swish")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        rn.linear_fwd(x, x, None, None, x)
    with pytest.raises(TypeError, match="CUDA"):
        rn.linear_gated_fwd(x, x, x, x)


# --------------------------------------------------------------------------
# the 64-bit definitions against differences
# --------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float64)


@pytest.mark.parametrize("act", sorted(rn.LINEAR_ACTS))
def test_gradients_against_differences(act):
    gen = torch.Generator().manual_seed(5)
    x, w, b, r, g = (_normal(gen, *s) for s in ((3, 16), (8, 16), (8,), (3, 8), (3, 8)))
    z = ref.linear_fwd(x, w, b, r, act)[0][1]
    loss = lambda: (ref.linear_fwd(x, w, b, r, act)[0][0] * g).sum()
    for got, at in zip(ref.linear_bwd(g, x, w, z, act, torch.float64)[0], (x, w, b)):
        torch.testing.assert_close(got, _differences(loss, at), rtol=1e-6, atol=1e-7)
    wu = _normal(gen, 8, 16)
    _, gate, up = ref.gated_fwd(x, w, wu, act)[0]
    loss = lambda: (ref.gated_fwd(x, w, wu, act)[0][0] * g).sum()
    for got, at in zip(ref.gated_bwd(g, x, w, wu, gate, up, act, torch.float64)[0], (x, w, wu)):
        torch.testing.assert_close(got, _differences(loss, at), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("act,fn", [("silu", torch.nn.functional.silu), ("sigmoid", torch.sigmoid), ("relu", torch.relu),
                                    ("gelu", torch.nn.functional.gelu),
                                    ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))])
def test_activations_are_the_usual_ones(act, fn):
    z = torch.linspace(-12, 12, 401, dtype=torch.float64, requires_grad=True)
    a = fn(z)
    slope, = torch.autograd.grad(a.sum(), z)
    (v, s), (ev, es) = ref.act(act, z.detach())
    torch.testing.assert_close(v, a.detach(), rtol=1e-9, atol=1e-12)
    torch.testing.assert_close(s, slope, rtol=1e-9, atol=1e-12)
    assert bool((ev <= 1e-4 * v.abs() + 1e-30).all()) and bool((es <= 1e-4).all())
