"""CPU checks of the operators around the mixers (fi_lattn_*, fi_dense_*,
fi_scores_*): the binding's structures have the header's layout, and every
create call refuses bad arguments before any device work."""
import ctypes
import os
import subprocess

import pytest

import exact_online_amd as fi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("fi_view", "fi_lattn_config", "fi_lattn_args", "fi_dense_config", "fi_dense_args", "fi_scores_config",
           "fi_scores_args")


def test_structures_match_the_header(tmp_path):
    lines, want = [], []
    for name in STRUCTS:
        C = getattr(fi, name)
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(C))
        for f, _ in C._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(C, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fi.h"\nint main(void) {' + "\n".join(lines) +
                   'printf("%d\\n", FI_SCORES_MAX_K); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True,
                   capture_output=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == want + [32]


INF, NAN = float("inf"), float("nan")
LATTN = dict(B=2, L=16, H=4, Hkv=2, dk=8, dv=8, scale=1.0, io_dtype=0, stream=None)
DENSE = dict(M=4, N=8, K=8, io_dtype=0, out_dtype=0, act=2, stream=None)
SCORES = dict(rows=4, V=100, k=5, io_dtype=0, scale=1.0, stream=None)
KINDS = {"lattn": (fi.fi_lattn_config, LATTN), "dense": (fi.fi_dense_config, DENSE),
         "scores": (fi.fi_scores_config, SCORES)}


def create(kind, **kw):
    C, base = KINDS[kind]
    cfg = C(**{**base, **kw})
    out = ctypes.c_void_p(123)
    fn = getattr(fi.lib, f"fi_{kind}_create")
    args = (ctypes.byref(cfg), 0x1000) if kind == "lattn" else (ctypes.byref(cfg),)   # a stand-in device pointer
    return fn(*args, ctypes.byref(out)), out.value


@pytest.mark.parametrize("kind,kw", [
    *[("lattn", {n: v}) for n in ("B", "L", "H", "Hkv", "dk", "dv") for v in (0, -1)],
    ("lattn", dict(Hkv=3)), ("lattn", dict(H=3)), ("lattn", dict(scale=INF)), ("lattn", dict(scale=NAN)),
    ("lattn", dict(io_dtype=2)), ("lattn", dict(io_dtype=-1)), ("lattn", dict(B=1 << 31)), ("lattn", dict(L=1 << 40)),
    ("lattn", dict(B=1 << 20, L=1 << 20, H=1 << 10)),
    *[("dense", {n: v}) for n in ("M", "N", "K") for v in (0, -5, 1 << 31)],
    ("dense", dict(io_dtype=7)), ("dense", dict(out_dtype=-1)), ("dense", dict(act=3)), ("dense", dict(act=-1)),
    *[("scores", {n: v}) for n in ("rows", "V") for v in (0, -1, 1 << 31)],
    ("scores", dict(k=-1)), ("scores", dict(k=33)), ("scores", dict(io_dtype=2)), ("scores", dict(scale=0.0)),
    ("scores", dict(scale=-1.0)), ("scores", dict(scale=NAN)), ("scores", dict(scale=INF)),
])
def test_create_refuses(kind, kw):
    assert create(kind, **kw) == (fi.FI_ERR_INVALID, None)


@pytest.mark.parametrize("kw", [dict(dk=257), dict(dv=1000), dict(L=fi.FI_MAX_L + 1), dict(B=1 << 20, H=2, Hkv=2)])
def test_lattn_create_unsupported_sizes(kw):
    assert create("lattn", **kw) == (fi.FI_ERR_UNSUPPORTED, None)


def test_null_arguments():
    out = ctypes.c_void_p(123)
    assert fi.lib.fi_lattn_create(None, 0x1000, ctypes.byref(out)) == fi.FI_ERR_INVALID and out.value is None
    cfg = fi.fi_lattn_config(**LATTN)
    assert fi.lib.fi_lattn_create(ctypes.byref(cfg), None, ctypes.byref(out)) == fi.FI_ERR_INVALID
    assert fi.lib.fi_lattn_create(ctypes.byref(cfg), 0x1000, None) == fi.FI_ERR_INVALID
    for kind in ("dense", "scores"):
        C, base = KINDS[kind]
        out = ctypes.c_void_p(123)
        fn = getattr(fi.lib, f"fi_{kind}_create")
        assert fn(None, ctypes.byref(out)) == fi.FI_ERR_INVALID and out.value is None
        assert fn(ctypes.byref(C(**base)), None) == fi.FI_ERR_INVALID
    assert fi.lib.fi_lattn_prompt(None, fi.fi_lattn_args()) == fi.FI_ERR_INVALID
    assert fi.lib.fi_lattn_step(None, fi.fi_lattn_args()) == fi.FI_ERR_INVALID
    assert fi.lib.fi_dense_run(None, fi.fi_dense_args()) == fi.FI_ERR_INVALID
    assert fi.lib.fi_scores_run(None, fi.fi_scores_args()) == fi.FI_ERR_INVALID
    for f in (fi.fi_lattn_destroy, fi.fi_dense_destroy, fi.fi_scores_destroy):
        f(None)


def test_create_without_gpu_is_unsupported():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for kind in KINDS:
        assert create(kind) == (fi.FI_ERR_UNSUPPORTED, None)
