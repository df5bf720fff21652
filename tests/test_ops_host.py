"""Refusals and no-ops of the stand-alone operators: no GPU needed, nothing launched."""
import ctypes as C

import numpy as np
import pytest

from tests import _ops_ref as ref

P = C.c_void_p(4096)       # an aligned address that is never followed


@pytest.fixture(scope="module")
def F():
    import fp4_expert_layer_b200 as F
    from fp4_expert_layer_b200 import build
    build.build()
    return F


def _args(base, **change):
    a = dict(base, **change)
    return list(a.values())


QUANT = dict(x=P, dtype=1, rows=8, K=64, ld=64, fmt=1, per=1, codes=P, scales=P, G=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(K=0), dict(K=48), dict(ld=63), dict(fmt=2), dict(fmt=-1),
    dict(per=0), dict(per=3), dict(x=None), dict(codes=None), dict(scales=None), dict(G=None),
    dict(codes=C.c_void_p(4097)), dict(x=C.c_void_p(4097)), dict(G=C.c_void_p(4098)),
    dict(rows=1 << 31, per=1), dict(rows=(1 << 31) - 1, K=1 << 20, ld=1 << 20),
])
def test_quantize_refuses(F, bad):
    L = F.lib()
    assert L.moe_fp4_quantize(*_args(QUANT, **bad)) == 1
    assert L.moe_last_error().startswith(b"moe_fp4_quantize")
    a = dict(QUANT, **bad)
    order = [a[n] for n in ("codes", "scales", "G", "fmt", "rows", "K", "per", "x", "dtype", "ld", "stream")]
    assert L.moe_fp4_dequantize(*order) == 1
    assert L.moe_last_error().startswith(b"moe_fp4_dequantize")


MATMUL = dict(xc=P, xs=P, xG=P, rows=4, wc=P, ws=P, wG=P, groups=2, N=8, K=64, fmt=1, offsets=P, y=P, dtype=1, ldy=8,
              stream=None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 27) + 1), dict(groups=0), dict(groups=1025), dict(N=0), dict(K=0), dict(K=40), dict(fmt=3), dict(dtype=3),
    dict(ldy=7), dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(y=None), dict(xG=None),
    dict(wG=None), dict(offsets=None), dict(xc=C.c_void_p(4104)), dict(wc=C.c_void_p(4104)), dict(y=C.c_void_p(4097)),
    dict(offsets=C.c_void_p(4098)), dict(groups=1024, N=1 << 21, ldy=1 << 21),
])
def test_matmul_refuses(F, bad):
    L = F.lib()
    assert L.moe_fp4_matmul(*_args(MATMUL, **bad)) == 1
    assert L.moe_last_error().startswith(b"moe_fp4_matmul")


@pytest.mark.parametrize("bad", [
    dict(N=(1 << 30) + 1, ldy=1 << 31), dict(N=(1 << 31) - 1, ldy=1 << 31), dict(K=(1 << 30) + 32),
    dict(K=(1 << 31) - 224), dict(K=(1 << 31) - 32),
])
def test_matmul_refuses_sizes_whose_tile_counts_overflow(F, bad):
    """One row, so that nothing else refuses them: a count of tiles or stages in 32 bits would be negative."""
    L = F.lib()
    assert L.moe_fp4_matmul(*_args(MATMUL, **dict(dict(rows=1, groups=1, N=1, ldy=1), **bad))) == 1
    assert b"2^30" in L.moe_last_error()


SORT = dict(ids=P, T=4, k=2, E=8, counts=P, offsets=P, perm=P, inv=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(ids=None), dict(counts=None),
    dict(offsets=None), dict(perm=None), dict(inv=None), dict(T=1 << 30, k=2),
])
def test_sort_refuses(F, bad):
    assert F.lib().moe_sort_tokens(*_args(SORT, **bad)) == 1


DISPATCH = dict(x=P, dtype=1, T=4, k=2, H=8, ldx=8, inv=P, rows=8, xs=P, ldxs=8, stream=None)
DBWD = dict(dxs=P, dtype=1, rows=8, T=4, k=2, H=8, lddxs=8, inv=P, dx=P, lddx=8, stream=None)
COMBINE = dict(ys=P, dti=1, rows=8, T=4, k=2, H=8, ldys=8, inv=P, gates=P, y=P, dto=0, ldy=8, stream=None)
CBWD = dict(dy=P, ddy=1, lddy=8, ys=P, dys_t=1, ldys=8, rows=8, T=4, k=2, H=8, inv=P, gates=P, dys=P, lddys=8, dg=P,
            stream=None)


@pytest.mark.parametrize("fn, base, bad", [
    ("moe_dispatch", DISPATCH, b) for b in (
        dict(dtype=4), dict(T=-1), dict(k=0), dict(k=33), dict(H=0), dict(H=(1 << 28) + 1, ldx=1 << 30, ldxs=1 << 30),
        dict(rows=-1), dict(ldx=7), dict(ldxs=7),
        dict(x=None), dict(inv=None), dict(xs=None), dict(x=C.c_void_p(4097)), dict(T=1 << 30, k=2))
] + [
    ("moe_dispatch_backward", DBWD, b) for b in (
        dict(dtype=3), dict(T=-1), dict(k=0), dict(H=0), dict(lddxs=7), dict(lddx=7), dict(dxs=None), dict(inv=None),
        dict(dx=None), dict(dx=C.c_void_p(4097)))
] + [
    ("moe_combine", COMBINE, b) for b in (
        dict(dti=3), dict(dto=3), dict(T=-1), dict(k=33), dict(rows=-1), dict(ldys=7), dict(ldy=7), dict(ys=None),
        dict(inv=None), dict(y=None), dict(y=C.c_void_p(4098)))
] + [
    ("moe_combine_backward", CBWD, b) for b in (
        dict(ddy=3), dict(dys_t=3), dict(T=-1), dict(k=0), dict(lddy=7), dict(ldys=7), dict(lddys=7), dict(dy=None),
        dict(ys=None), dict(inv=None), dict(dys=None, dg=None), dict(dys=C.c_void_p(4097)))
])
def test_row_operators_refuse(F, fn, base, bad):
    assert getattr(F.lib(), fn)(*_args(base, **bad)) == 1
    assert F.lib().moe_last_error().startswith(fn.encode())


@pytest.mark.parametrize("fn, base, empty", [
    ("moe_fp4_quantize", QUANT, dict(rows=0, x=None, codes=None, scales=None, G=None)),
    ("moe_fp4_matmul", MATMUL, dict(rows=0, xc=None, xs=None, xG=None, y=None)),
    ("moe_dispatch", DISPATCH, dict(T=0, x=None, inv=None)),
    ("moe_dispatch", DISPATCH, dict(rows=0, xs=None)),
    ("moe_dispatch_backward", DBWD, dict(T=0, dx=None)),
    ("moe_combine", COMBINE, dict(T=0, y=None)),
    ("moe_combine_backward", CBWD, dict(T=0, dy=None, dys=None, dg=None)),
])
def test_nothing_to_do_is_a_no_op(F, fn, base, empty):
    assert getattr(F.lib(), fn)(*_args(base, **empty)) == 0


def test_binding_refuses_before_the_library(F):
    import torch
    x = torch.zeros((4, 64))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: F.fp4_quantize(x), lambda: F.sort_tokens(ids, 8), lambda: F.dispatch(x, ids),
                 lambda: F.combine(x, ids), lambda: F.dispatch_backward(x, ids),
                 lambda: F.combine_backward(x, x, ids)):
        with pytest.raises(F.MoEError) as ei:
            call()
        assert ei.value.status == 1 and "CUDA" in str(ei.value)


def test_definitions_agree_with_the_oracles_tables():
    """The numpy definitions against the C oracle's decoders, code by code."""
    import oracle
    L = oracle.lib()
    for c in range(16):
        v = (-1.0 if c & 8 else 1.0) * ref.E2M1[c & 7]
        assert L.orc_e2m1(c) == v
    for c in range(1, 255):
        assert L.orc_e8m0(c) == 2.0 ** (c - 127)
    tab = ref.e4m3_table()
    assert np.all(np.diff(tab) > 0) and tab[126] == 448.0 and tab[8] == 2.0 ** -6 and tab[1] == 2.0 ** -9


def test_definition_of_a_tie():
    """Codes on a border go to the even one; scales likewise."""
    x = np.array([[6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] + [-.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0] + [0] * 16])
    c, s, _, v = ref.quantize(x, "mxfp4")
    assert s[0, 0] == 127
    assert v[0, :16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -1, -2, -2, -4, -4, 0]


# ------------------------------------------------------------------ the build
def _build_in_a_child(tmp_path, setup, path=()):
    """What build.build() returns with the binding's file elsewhere; the library is up to date."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = f"from fp4_expert_layer_b200 import build as b\nb.SO_BINDING = {str(tmp_path / '_ops.so')!r}\n{setup}\nprint(b.build())"
    env = {k: v for k, v in os.environ.items() if k not in ("CUDA_HOME", "CUDA_PATH")}
    env["PYTHONPATH"] = os.pathsep.join([*map(str, path), root])
    return subprocess.run([sys.executable, "-c", code], cwd=root, env=env, capture_output=True, text=True, timeout=600)


def test_the_library_builds_beside_a_torch_without_cuda(F, tmp_path):
    t = tmp_path / "torch"
    t.mkdir()
    for name in ("__init__.py", "version.py"):
        (t / name).write_text("__version__ = '9.9.0+cpu'\ncuda = None\n")
    r = _build_in_a_child(tmp_path, "", [tmp_path])
    assert r.returncode == 0 and r.stdout.strip().endswith("libfp4moe.so"), r.stderr[-2000:]
    assert not (tmp_path / "_ops.so").exists()


def test_the_library_builds_where_the_binding_has_no_toolkit(F, tmp_path):
    r = _build_in_a_child(tmp_path, "b.shutil.which = lambda name: None\nb.CUDA_ROOTS = ()")
    assert r.returncode == 0 and r.stdout.strip().endswith("libfp4moe.so"), r.stderr[-2000:]
    assert "binding is not built" in r.stderr and not (tmp_path / "_ops.so").exists()


def test_a_binding_that_fails_to_compile_leaves_a_built_library(F, tmp_path):
    """The library comes first, and the failure is not kept quiet."""
    r = _build_in_a_child(tmp_path, "\n".join((
        "import subprocess", "made = []",
        "def run(cmd, check):",
        "    made.append(cmd[0])",
        "    if cmd[0] == 'g++': raise subprocess.CalledProcessError(1, cmd)",
        "    open(cmd[cmd.index('-o') + 1], 'w').close()",
        "b.subprocess.run = run", f"b.SO = {str(tmp_path / 'lib.so')!r}",
        "import atexit; atexit.register(lambda: print(made))")))
    assert r.returncode != 0 and "CalledProcessError" in r.stderr
    assert "['nvcc', 'g++']" in r.stdout and (tmp_path / "lib.so").exists()


def test_a_binding_of_another_torch_or_python_is_built_again(F, tmp_path, monkeypatch):
    import os
    from fp4_expert_layer_b200 import build as b
    made = []

    def compiled(cmd, check):
        made.append(next(c for c in cmd if "MOE_TORCH_VERSION" in c))
        open(cmd[cmd.index("-o") + 1], "w").close()

    here = b._torch()
    monkeypatch.setattr(b, "SO_BINDING", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(b.subprocess, "run", compiled)
    assert b.build_binding() == b.SO_BINDING and b.build_binding() == b.SO_BINDING
    assert len(made) == 1 and here[0] in made[0]
    monkeypatch.setattr(b, "_torch", lambda: ("9.9.0", *here[1:]))
    b.build_binding(), b.build_binding()
    assert len(made) == 2 and "9.9.0" in made[1]
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399")
    b.build_binding(), b.build_binding()
    assert len(made) == 3
    os.remove(b.SO_BINDING)
    b.build_binding()
    assert len(made) == 4


def test_arguments_of_another_kind_are_refused_beside_a_stream_too(F):
    """The detour of calls with stream= looks at the arguments before the compiled check does."""
    import torch
    x, ids = torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int32)
    for stream in (None, 0, 1):
        for call in (lambda s: F.fp4_quantize("x", stream=s), lambda s: F.fp4_dequantize(None, stream=s),
                     lambda s: F.fp4_dequantize((), stream=s), lambda s: F.fp4_matmul(None, None, stream=s),
                     lambda s: F.fp4_matmul(x, None, stream=s), lambda s: F.fp4_matmul((None,) * 4, 7, stream=s),
                     lambda s: F.sort_tokens([1, 2], 4, stream=s), lambda s: F.dispatch(None, ids, stream=s),
                     lambda s: F.dispatch_backward(3, ids, stream=s), lambda s: F.combine("x", ids, stream=s),
                     lambda s: F.combine_backward(None, x, ids, stream=s), lambda s: F.fp4_quantize(x, out=3, stream=s)):
            with pytest.raises(F.MoEError) as ei:
                call(stream)
            assert ei.value.status == 1
