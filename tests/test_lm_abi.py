"""The C ABI of the operators around the scan on the CPU: struct layouts and host-side
validation, with fake device addresses that nothing dereferences (the entry points return before
any HIP call)."""
import ctypes
import os
import subprocess

import pytest

from selective_state_space_26_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS, ALIAS, VERSION = 0, 1, 2, 3, 4, 5, 6, 7, 9
STRUCTS = {"msel_norm_args": _lib.NormArgs, "msel_norm_grads": _lib.NormGrads,
           "msel_gated_norm_args": _lib.GatedNormArgs,
           "msel_gated_norm_grads": _lib.GatedNormGrads, "msel_embed_args": _lib.EmbedArgs,
           "msel_embed_grads": _lib.EmbedGrads, "msel_tensor": _lib.TensorEntry,
           "msel_grad_args": _lib.GradArgs}

_fake = iter(range(0x10000000, 0x7fffffff, 0x100000))


def _addr():
    return next(_fake)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_struct_layout_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    body = "".join(f'printf("{n} %zu\\n", sizeof({n}));\n'
                   + "".join(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));\n'
                             for f, _ in s._fields_) for n, s in STRUCTS.items())
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "msel.h"\n'
                   "int main(void) {\n" + body + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out.strip().splitlines())}
    for n, s in STRUCTS.items():
        assert got[n] == ctypes.sizeof(s), n
        for f, _ in s._fields_:
            assert got[f"{n}.{f}"] == getattr(s, f).offset, (n, f)


def _norm(**kw):
    a = _lib.NormArgs(1, 100, 7, 1, 0, 1.0, 1e-5, _addr(), _addr(), _addr(), _addr(), _addr())
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _norm_grads(**kw):
    g = _lib.NormGrads(*[_addr() for _ in range(6)])
    for k, v in kw.items():
        setattr(g, k, v)
    return g


NAN = float("nan")


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(residual=None), OK), (dict(weight=None), OK), (dict(residual_out=None), OK),
    (dict(residual_dtype=1), OK), (dict(eps=0.0), OK), (dict(dim=16384), OK),
    (dict(abi_version=2), VERSION), (dict(dim=0), SHAPE), (dict(rows=0), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 40), SHAPE), (dict(rows=2 ** 62, dim=4), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(dim=16385), UNSUP), (dict(dtype=2), DTYPE), (dict(residual_dtype=7), DTYPE),
    (dict(dtype=0, residual_dtype=1), DTYPE), (dict(x=None), NULL), (dict(out=None), NULL),
    (dict(x=0x1008), ALIGN), (dict(residual=0x1008), ALIGN), (dict(out=0x1008), ALIGN),
    (dict(residual_out=0x1008), ALIGN), (dict(weight=0x1002), ALIGN)])
def test_norm_fwd_checks(lib, kw, code):
    assert lib.msel_validate_norm_fwd(ctypes.byref(_norm(**kw))) == code


@pytest.mark.parametrize("out,of,code", [
    ("out", "x", ALIAS), ("out", "residual", ALIAS), ("out", "weight", ALIAS),
    ("out", "residual_out", ALIAS), ("residual_out", "x", ALIAS),
    ("residual_out", "weight", ALIAS), ("residual_out", "residual", OK)])
def test_norm_fwd_aliases(lib, out, of, code):
    a = _norm()
    setattr(a, out, getattr(a, of))
    assert lib.msel_validate_norm_fwd(ctypes.byref(a)) == code


def test_norm_bwd_checks(lib):
    a, ws = _norm(x=None, residual=None, out=None, residual_out=None), _addr()
    need = lib.msel_norm_bwd_workspace_bytes(ctypes.byref(a))
    assert need > 0 and need % (4 * a.dim) == 0
    assert lib.msel_norm_bwd_workspace_bytes(ctypes.byref(_norm(dim=0))) == 0

    def v(g, w=ws, n=need):
        return lib.msel_validate_norm_bwd(ctypes.byref(a), ctypes.byref(g) if g else None, w, n)
    assert v(_norm_grads()) == OK
    assert v(None) == NULL
    assert v(_norm_grads(s=None)) == NULL
    assert v(_norm_grads(dout=None)) == NULL
    assert v(_norm_grads(dx=None, dresidual=None, dweight=None)) == NULL
    assert v(_norm_grads(dresidual_out=None)) == OK
    assert v(_norm_grads(dweight=None), None, 0) == OK
    assert v(_norm_grads(), None, need) == WS
    assert v(_norm_grads(), ws, need - 1) == WS
    assert v(_norm_grads(), ws + 16, need) == ALIGN
    assert v(_norm_grads(dx=0x1008)) == ALIGN
    assert v(_norm_grads(dweight=0x1001)) == ALIGN
    for out in ("dx", "dweight", "dresidual"):
        for of in ("s", "dout"):
            g = _norm_grads()
            setattr(g, out, getattr(g, of))
            assert v(g) == ALIAS, (out, of)
    g = _norm_grads()
    g.dresidual = g.dresidual_out
    assert v(g) == OK
    g.dx = g.dresidual
    assert v(g) == ALIAS
    assert v(_norm_grads(s=ws)) == ALIAS


def _gated(**kw):
    a = _lib.GatedNormArgs(1, 2, 96, 50, 2, 1, 0, 1, 1, 1e-5, _addr(), _addr(), _addr(), _addr())
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(weight=None), OK), (dict(layout=1), OK), (dict(out_layout=0), OK),
    (dict(abi_version=0), VERSION), (dict(batch=0), SHAPE), (dict(dim=0), SHAPE),
    (dict(seqlen=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE),
    (dict(batch=1 << 30), SHAPE), (dict(seqlen=(1 << 28) + 1), SHAPE),
    (dict(batch=1 << 10, seqlen=1 << 28), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(dim=16385, groups=1), UNSUP), (dict(dim=32768, groups=2), OK),
    (dict(dim=4096, groups=2048), UNSUP), (dict(layout=1, out_layout=0), UNSUP),
    (dict(dtype=3), DTYPE), (dict(layout=2), DTYPE), (dict(out_layout=-1), DTYPE),
    (dict(gate_first=2), DTYPE), (dict(x=None), NULL), (dict(z=None), NULL),
    (dict(out=None), NULL), (dict(x=0x1004), ALIGN), (dict(z=0x1004), ALIGN),
    (dict(out=0x1004), ALIGN), (dict(weight=0x1001), ALIGN)])
def test_gated_fwd_checks(lib, kw, code):
    assert lib.msel_validate_gated_norm_fwd(ctypes.byref(_gated(**kw))) == code


def test_gated_bwd_checks(lib):
    for kw in ({}, dict(layout=1), dict(seqlen=1), dict(dtype=0), dict(gate_first=0)):
        a, ws = _gated(**kw), _addr()
        need = lib.msel_gated_norm_bwd_workspace_bytes(ctypes.byref(a))
        assert need > 0 and need % (4 * a.dim) == 0

        def v(g, w=ws, n=need):
            return lib.msel_validate_gated_norm_bwd(ctypes.byref(a), ctypes.byref(g), w, n)

        def grads():
            return _lib.GatedNormGrads(*[_addr() for _ in range(4)])
        assert v(grads()) == OK
        for f in ("dout", "dx", "dz"):
            g = grads()
            setattr(g, f, None)
            assert v(g) == NULL
            setattr(g, f, 0x1008)
            assert v(g) == ALIGN
        g = grads()
        assert v(g, ws, need - 1) == WS and v(g, None, need) == WS
        g.dweight = None
        assert v(g, None, 0) == OK
        for out in ("dx", "dz", "dweight"):
            for of in (a.x, a.z, a.weight):
                g = grads()
                setattr(g, out, of)
                assert v(g) == ALIAS
        g = grads()
        g.dz = g.dx
        assert v(g) == ALIAS
    a = _gated()
    a.out = a.z
    assert lib.msel_validate_gated_norm_fwd(ctypes.byref(a)) == ALIAS


def _embed(**kw):
    a = _lib.EmbedArgs(1, 1000, 64, 1, 300, -1, 1, 0, 1.0, 0, _addr(), _addr(), _addr())
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(ids_64bit=0), OK), (dict(padding_idx=1 << 40), OK),
    (dict(abi_version=2), VERSION), (dict(reserved=1), VERSION), (dict(vocab=0), SHAPE),
    (dict(dim=0), SHAPE), (dict(tokens=0), SHAPE), (dict(tokens=(1 << 30) + 1), SHAPE),
    (dict(vocab=(1 << 30) + 1), SHAPE), (dict(vocab=1 << 30, dim=2048), SHAPE),
    (dict(dim=16385), UNSUP), (dict(dtype=2), DTYPE), (dict(weight_dtype=2), DTYPE),
    (dict(ids_64bit=2), DTYPE), (dict(ids=None), NULL), (dict(weight=None), NULL),
    (dict(out=None), NULL), (dict(ids=0x1004), ALIGN), (dict(weight=0x1008), ALIGN),
    (dict(out=0x1008), ALIGN)])
def test_embed_fwd_checks(lib, kw, code):
    assert lib.msel_validate_embed_fwd(ctypes.byref(_embed(**kw))) == code


def test_embed_bwd_checks(lib):
    a, ws = _embed(weight=None, out=None), _addr()
    need = lib.msel_embed_bwd_workspace_bytes(ctypes.byref(a))
    assert need >= 4 * 4 * 300
    assert lib.msel_embed_bwd_workspace_bytes(ctypes.byref(_embed(dim=0))) == 0

    def v(g, w=ws, n=need):
        return lib.msel_validate_embed_bwd(ctypes.byref(a), ctypes.byref(g), w, n)
    good = _lib.EmbedGrads(_addr(), _addr(), _addr())
    assert v(good) == OK
    assert v(_lib.EmbedGrads(good.dout, None, good.dweight)) == OK
    assert v(_lib.EmbedGrads(good.dout, good.dweight, good.dweight)) == OK
    assert v(_lib.EmbedGrads(None, None, good.dweight)) == NULL
    assert v(_lib.EmbedGrads(good.dout, None, None)) == NULL
    assert v(_lib.EmbedGrads(good.dout, None, good.dout)) == ALIAS
    assert v(_lib.EmbedGrads(good.dout, None, a.ids)) == ALIAS
    assert v(_lib.EmbedGrads(good.dout + 8, None, good.dweight)) == ALIGN
    assert v(_lib.EmbedGrads(good.dout, good.base + 4, good.dweight)) == ALIGN
    assert v(good, None, need) == WS and v(good, ws, need - 1) == WS
    assert v(good, ws + 128, need) == ALIGN
    assert v(good, good.dout, need) == ALIAS


def _entries(*items):
    e = (_lib.TensorEntry * len(items))()
    for i, (data, n, dt) in enumerate(items):
        e[i] = _lib.TensorEntry(data, n, dt, 0)
    return e


def test_grad_checks(lib):
    p, q, norm, ws = _addr(), _addr(), _addr(), _addr()
    e = _entries((p, 1000, 0), (q, 77, 1), (None, 0, 0))

    def args(entries=e, outs=e, count=None, **kw):
        a = _lib.GradArgs(1, len(entries) if count is None else count, entries, outs, 1.0, 1e-6,
                          norm)
        for k, v in kw.items():
            setattr(a, k, v)
        return a
    need = lib.msel_grad_workspace_bytes(ctypes.byref(args()))
    assert need == 3 * 8  # two chunks and the factor

    def v(a, w=ws, n=need):
        return lib.msel_validate_grad_clip(ctypes.byref(a), w, n)
    assert v(args()) == OK
    assert lib.msel_validate_grad_norm(ctypes.byref(args(outs=None)), ws, need) == OK
    assert v(args(count=0), ws, 8) == OK
    assert v(args(abi_version=3)) == VERSION
    assert v(args(count=-1)) == SHAPE
    assert v(args(outs=None)) == NULL
    assert v(args(norm=None)) == NULL
    assert v(args(norm=norm + 2)) == ALIGN
    assert v(args(max_norm=-1.0)) == SHAPE and v(args(max_norm=NAN)) == SHAPE
    assert v(args(max_norm=float("inf"))) == OK
    assert v(args(eps=-1.0)) == SHAPE
    assert v(args(), None, need) == WS and v(args(), ws, need - 8) == WS
    assert v(args(), ws + 8, need) == ALIGN
    assert v(args(norm=p)) == ALIAS and v(args(), p, need) == ALIAS
    for bad, code in (((p, -1, 0), SHAPE), ((p, (1 << 40) + 1, 0), SHAPE), ((p, 5, 2), DTYPE),
                      ((None, 5, 0), NULL), ((p + 2, 5, 0), ALIGN), ((p + 1, 5, 1), ALIGN)):
        b = _entries(bad)
        assert v(args(b, b)) == code, bad
    b = _entries((p, 1000, 0), (q, 78, 1), (None, 0, 0))
    assert v(args(outs=b)) == SHAPE
    b = _entries((p, 1000, 0), (q, 77, 0), (None, 0, 0))
    assert v(args(outs=b)) == DTYPE
    b = _entries((p, 1000, 0), (norm, 77, 1), (None, 0, 0))
    assert v(args(outs=b)) == ALIAS


def test_null_argument_pointers(lib):
    for fn in ("msel_validate_norm_fwd", "msel_validate_gated_norm_fwd",
               "msel_validate_embed_fwd"):
        assert getattr(lib, fn)(None) == NULL
    for fn in ("msel_validate_norm_bwd", "msel_validate_gated_norm_bwd",
               "msel_validate_embed_bwd"):
        assert getattr(lib, fn)(None, None, None, 0) == NULL
    for fn in ("msel_validate_grad_norm", "msel_validate_grad_clip"):
        assert getattr(lib, fn)(None, None, 0) == NULL
    # the entry points themselves, before any HIP call
    assert lib.msel_norm_fwd(None, None) == NULL
    assert lib.msel_gated_norm_bwd(None, None, None, 0, None) == NULL
    assert lib.msel_embed_bwd(None, None, None, 0, None) == NULL
    assert lib.msel_grad_clip(None, None, 0, None) == NULL


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import selective_state_space_26_amd as msel
    x = torch.zeros(2, 4, 8)
    ids = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: msel.msel_norm_fwd(x), lambda: msel.msel_norm_bwd(x, None, x),
                 lambda: msel.msel_gated_norm_fwd(x, x),
                 lambda: msel.msel_gated_norm_bwd(x, x, None, x),
                 lambda: msel.msel_embed_fwd(ids, x[0]),
                 lambda: msel.msel_embed_bwd(ids, x[0, :3], 4),
                 lambda: msel.msel_grad_norm([x]), lambda: msel.msel_grad_clip([x], 1.0)):
        with pytest.raises(ValueError):
            call()
