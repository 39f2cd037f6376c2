"""Sanitizer run of the operators' host code (CPU only, no GPU needed).

The library's host side, with clang's AddressSanitizer and
UndefinedBehaviorSanitizer, without device code (an empty code object stands in
for it: nothing is launched on a machine without a device).  A child process under
the sanitizer runtime calls every entry point of fi_lattn_*, fi_dense_* and
fi_scores_*: create calls that are refused, calls on handles in host
memory that are refused, and calls that are planned and go as far as the launch,
over many sizes.  It must exit 0 with no sanitizer report.
"""
import os
import re
import subprocess
import sys
from pathlib import Path

import pytest

import test_sanitize_cpu as san

ROOT = san.ROOT

PROBE = r'''
import ctypes, itertools, random, sys
sys.modules["torch"] = None            # the binding alone
sys.path.insert(0, sys.argv[1])
import exact_online_amd as fi
INVALID, NO_DEVICE = fi.FI_ERR_INVALID, (fi.FI_ERR_UNSUPPORTED, fi.FI_ERR_HIP)
lib, P, rng = fi.lib, 4096, random.Random(3)    # P: a stand-in device pointer, never dereferenced here
calls = 0

def check(got, want, what):
    global calls
    calls += 1
    assert got in (want if isinstance(want, tuple) else (want,)), (what, got)

def create(kind, want, *before, **kw):
    out = ctypes.c_void_p(1)
    cfg = getattr(fi, f"fi_{kind}_config")(**kw)
    args = (P,) if kind == "lattn" else ()
    check(getattr(lib, f"fi_{kind}_create")(ctypes.byref(cfg), *args, ctypes.byref(out)), want, (kind, kw))
    assert out.value is None
    return cfg

BASE = dict(lattn=dict(B=2, L=16, H=4, Hkv=2, dk=8, dv=8, scale=1.0), dense=dict(M=4, N=8, K=8, act=2),
            scores=dict(rows=4, V=100, k=5, scale=1.0))
EDGES = (0, -1, 1 << 31, 1 << 40, (1 << 63) - 1, -(1 << 63))
for kind, base in BASE.items():
    fn = getattr(lib, f"fi_{kind}_create")
    out = ctypes.c_void_p(1)
    dev = (P,) if kind == "lattn" else ()
    check(fn(None, *dev, ctypes.byref(out)), INVALID, kind)
    check(fn(ctypes.byref(getattr(fi, f"fi_{kind}_config")(**base)), *dev, None), INVALID, kind)
    create(kind, NO_DEVICE, **base)
    for name in base:
        if name in ("scale", "act", "k"):
            continue
        for v in EDGES:
            create(kind, (INVALID, fi.FI_ERR_UNSUPPORTED), **{**base, name: v})
    for dt in (2, -1, 1 << 30, -(1 << 31)):
        create(kind, INVALID, **{**base, "io_dtype": dt})
    for s in (0.0, -1.0, float("inf"), float("nan")):
        if kind == "scores":
            create(kind, INVALID, **{**base, "scale": s})
create("lattn", fi.FI_ERR_UNSUPPORTED, **{**BASE["lattn"], "dk": 257})
create("dense", INVALID, **{**BASE["dense"], "act": 9})
create("dense", INVALID, **{**BASE["dense"], "out_dtype": 5})
create("scores", INVALID, **{**BASE["scores"], "k": 33})
for f in (lib.fi_lattn_destroy, lib.fi_dense_destroy, lib.fi_scores_destroy):
    f(None)

# handles as the create calls lay them out
def handle(cfg, *more):
    class H(ctypes.Structure):
        _fields_ = [("cfg", type(cfg)), ("stream", ctypes.c_void_p)] + [(f"p{i}", ctypes.c_void_p) for i in range(len(more))]
    return H(cfg, None, *more)

def spread(lo, hi):
    return int(lo * (hi / lo) ** rng.random())

for i in range(3000):
    io, od = rng.choice((0, 1)), rng.choice((0, 1))
    # linear attention
    Hkv, G, dk, dv = rng.randint(1, 20), rng.randint(1, 9), rng.randint(1, 256), rng.randint(1, 256)
    B, L = spread(1, 4000), spread(1, 100000)
    h = handle(fi.fi_lattn_config(B=B, L=L, H=Hkv * G, Hkv=Hkv, dk=dk, dv=dv, scale=1.0, io_dtype=io), P, P)
    b, l = rng.choice((B, 1, spread(1, B), 0)), rng.choice((L, 1, spread(1, L), 0))
    big = 1 << rng.randint(0, 50)
    v = lambda: fi.fi_view(P, rng.choice((l * Hkv * dk, 0, -big, big)), rng.choice((Hkv * dk, 0, -big, big)), rng.choice((dk, 0, -big, big)))
    ok = dict(B=b, L=l, q=v(), k=v(), v=v(), o=v(), lens=rng.choice((0, P)), slots=rng.choice((0, P)), n_slots=b + rng.randint(0, 5),
              state=P, fresh=rng.choice((0, 1)))
    call = lambda name, **kw: getattr(lib, f"fi_lattn_{name}")(ctypes.addressof(h), fi.fi_lattn_args(**{**ok, **kw}))
    ran = fi.FI_OK if b == 0 else NO_DEVICE
    check(call("prompt"), ran, ok)
    check(call("step", lens=0, L=1), ran, ok)
    check(call("prompt", state=0, fresh=1), ran, ok)
    for kw in (dict(B=B + 1), dict(B=-1), dict(L=L + 1), dict(L=-1), dict(n_slots=-1), dict(n_slots=1 << 31), dict(state=P + 4),
               dict(lens=P + 2), dict(slots=P + 1), dict(state=0, fresh=0), dict(q=fi.fi_view(P + 1, 0, 0, 0))):
        check(call("prompt", **kw), INVALID, kw)
    check(call("step", L=2), INVALID, "L")
    check(call("step", L=1, lens=P), INVALID, "lens")
    if b:
        check(call("step", L=1, lens=0, state=0, fresh=1), INVALID, "state")
    # dense product
    M, N, K = spread(1, 1 << 20), spread(1, 60000), spread(1, 60000)
    h2 = handle(fi.fi_dense_config(M=M, N=N, K=K, io_dtype=io, out_dtype=od, act=rng.choice((0, 1, 2))), P)
    m = rng.choice((M, 1, spread(1, M), 0))
    ok2 = dict(M=m, x=P, ldx=K + rng.choice((0, 1, 64)), w=P, ldw=K, bias=rng.choice((0, P)), res=rng.choice((0, P)), ldr=N, y=P, ldy=N)
    call2 = lambda **kw: lib.fi_dense_run(ctypes.addressof(h2), fi.fi_dense_args(**{**ok2, **kw}))
    check(call2(), fi.FI_OK if m == 0 else NO_DEVICE, ok2)
    for kw in (dict(M=M + 1), dict(M=-1)) + ((dict(x=0), dict(w=0), dict(y=0), dict(ldx=K - 1), dict(ldw=-1), dict(ldy=N - 1),
               dict(res=P, ldr=N - 1), dict(ldx=1 << 62), dict(x=P + 1), dict(y=P + 1), dict(bias=P + 1)) if m else ()):
        check(call2(**kw), INVALID, kw)
    # token scores
    R, V, k = spread(1, 1 << 20), spread(1, 1 << 24), rng.randint(0, 32)
    h3 = handle(fi.fi_scores_config(rows=R, V=V, k=k, io_dtype=io, scale=1.0), P, P)
    r = rng.choice((R, 1, spread(1, R), 0))
    ok3 = dict(rows=r, logits=P, ld=V + rng.choice((0, 7)), targets=P, logprob=P, entropy=rng.choice((0, P)), lse=rng.choice((0, P)),
               top=P, top_id=P)
    call3 = lambda **kw: lib.fi_scores_run(ctypes.addressof(h3), fi.fi_scores_args(**{**ok3, **kw}))
    check(call3(), fi.FI_OK if r == 0 else NO_DEVICE, ok3)
    for kw in (dict(rows=R + 1), dict(rows=-1)) + ((dict(logits=0), dict(ld=V - 1), dict(ld=1 << 62), dict(targets=0), dict(logprob=0),
               dict(logits=P + 1), dict(targets=P + 4), dict(top_id=P + 4), dict(entropy=P + 2)) if r else ()):
        check(call3(**kw), INVALID, kw)
for f in (lib.fi_lattn_prompt, lib.fi_lattn_step, lib.fi_dense_run, lib.fi_scores_run):
    check(f(None, f.argtypes[1]._type_()), INVALID, f)
for f, x in ((lib.fi_lattn_prompt, h), (lib.fi_lattn_step, h), (lib.fi_dense_run, h2), (lib.fi_scores_run, h3)):
    check(f(ctypes.addressof(x), None), INVALID, f)
print("probe ok", calls)
'''


@pytest.mark.skipif(not Path(san.HIPCC).exists(), reason="hipcc missing")
def test_operators_host_code_under_asan_ubsan(tmp_path):
    if os.path.exists("/dev/kfd"):
        pytest.skip("the handles are not of this machine's device")
    rt = san._asan_runtime()
    if rt is None:
        pytest.skip("clang's AddressSanitizer runtime is missing")
    sys.path.insert(0, str(ROOT / "exact_online_amd"))
    import build as fib
    flags = [f for f in fib.FLAGS if f != "-O3"] + ["-O1", "-g", "--offload-host-only", f"-I{ROOT / 'include'}", f"-I{fib.CSRC}"]
    for f in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer"):
        flags += ["-Xarch_host", f]
    objs = []
    for src in fib.SOURCES:
        objs.append(str(tmp_path / (src.name + ".o")))
        subprocess.run([fib.HIPCC, *flags, "-c", str(src), "-o", objs[-1]], check=True, capture_output=True, text=True)
    # the code objects that the host side registers
    names = set(re.findall(r"\bU (__hip_fatbin\w*)", subprocess.run(["nm", *objs], check=True, capture_output=True, text=True).stdout))
    stub = tmp_path / "no_code.c"
    stub.write_text("".join(f"const char {n}[4096] __attribute__((aligned(4096))) = {{0}};\n" for n in sorted(names)))
    subprocess.run(["gcc", "-fPIC", "-c", str(stub), "-o", str(tmp_path / "no_code.o")], check=True)
    lib = tmp_path / "libfi_asan.so"
    subprocess.run([fib.HIPCC, *flags, "-shared", "-o", str(lib), *objs, str(tmp_path / "no_code.o")], check=True,
                   capture_output=True, text=True)
    probe = tmp_path / "probe.py"
    probe.write_text(PROBE)
    env = dict(os.environ, LD_PRELOAD=str(rt), ASAN_OPTIONS="detect_leaks=0", EXACT_ONLINE_AMD_LIB=str(lib))
    r = subprocess.run([sys.executable, str(probe), str(ROOT)], capture_output=True, text=True, timeout=300, env=env)
    san._no_report(r)
    assert "probe ok" in r.stdout
