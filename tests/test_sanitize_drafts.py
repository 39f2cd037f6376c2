"""Sanitizer run of the host code of fi_delta_*, fi_rotary_* and fi_verify_* (CPU only), as
test_sanitize_operators.py does it for the other operators: the library's host side
with clang's AddressSanitizer and UndefinedBehaviorSanitizer and an empty code object, calls
on handles in host memory that are refused, and ones that are planned and go as far as the launch."""
import os
import re
import subprocess
import sys
from pathlib import Path

import pytest

import test_sanitize_cpu as san

ROOT = san.ROOT

PROBE = r'''
import ctypes, random, sys
sys.modules["torch"] = None            # the binding alone
sys.path.insert(0, sys.argv[1])
import exact_online_amd as fi
INVALID, NO_DEVICE = fi.FI_ERR_INVALID, (fi.FI_ERR_UNSUPPORTED, fi.FI_ERR_HIP)
lib, P, rng = fi.lib, 4096, random.Random(5)    # P: a stand-in device pointer, never dereferenced here
calls = 0

def check(got, want, what):
    global calls
    calls += 1
    assert got in (want if isinstance(want, tuple) else (want,)), (what, got)

BASE = dict(delta=dict(B=2, L=16, Hk=2, Hv=4, dk=8, dv=8, scale=1.0), rotary=dict(B=2, L=16, Hq=4, Hk=2, d=8, rot=8, norm=1, eps=1e-6),
            verify=dict(B=2, N=3, V=100, scale=1.0, draft_scale=1.0))
for kind, base in BASE.items():
    fn, C = getattr(lib, f"fi_{kind}_create"), getattr(fi, f"fi_{kind}_config")
    dev = (P,) if kind == "rotary" else ()
    def create(want, **kw):
        out = ctypes.c_void_p(1)
        check(fn(ctypes.byref(C(**{**base, **kw})), *dev, ctypes.byref(out)), want, (kind, kw))
        assert out.value is None
    create(NO_DEVICE)
    for name in base:
        if name in ("scale", "draft_scale", "eps"):
            for x in (float("nan"), float("inf"), -1.0) if name != "scale" or kind != "delta" else (float("nan"),):
                create(INVALID, **{name: x})
            continue
        for v in (-1, 1 << 31, 1 << 40, (1 << 63) - 1, -(1 << 63)):
            if name != "norm":
                create((INVALID, fi.FI_ERR_UNSUPPORTED), **{name: v})
    for dt in (2, -1, 1 << 30, -(1 << 31)):
        create(INVALID, io_dtype=dt)
    getattr(lib, f"fi_{kind}_destroy")(None)

def handle(cfg):
    class H(ctypes.Structure):
        _fields_ = [("cfg", type(cfg)), ("stream", ctypes.c_void_p), ("device", ctypes.c_int), ("p", ctypes.c_void_p * 4)]
    return H(cfg, None, 0, (ctypes.c_void_p * 4)(P, P, P, P))

def spread(lo, hi):
    return int(lo * (hi / lo) ** rng.random())

for i in range(3000):
    io = rng.choice((0, 1))
    Hk, G, dk, dv = rng.randint(1, 20), rng.randint(1, 9), rng.randint(1, 256), rng.randint(1, 256)
    B, L = spread(1, 4000), spread(1, 100000)
    h = handle(fi.fi_delta_config(B=B, L=L, Hk=Hk, Hv=Hk * G, dk=dk, dv=dv, scale=1.0, io_dtype=io))
    b, l, big = rng.choice((B, 1, spread(1, B), 0)), rng.choice((L, 1, spread(1, L), 0)), 1 << rng.randint(0, 50)
    v = lambda: fi.fi_view(P, rng.choice((l * Hk * dk, 0, -big, big)), rng.choice((Hk * dk, 0, -big, big)), rng.choice((dk, 0, -big, big)))
    ok = dict(B=b, L=l, q=v(), k=v(), v=v(), o=v(), log_decay=v(), beta=v(), lens=rng.choice((0, P)), slots=rng.choice((0, P)),
              n_slots=b + rng.randint(0, 5), state=P, fresh=rng.choice((0, 1)), hold=rng.choice((0, 1, -7)))
    call = lambda name, **kw: getattr(lib, f"fi_delta_{name}")(ctypes.addressof(h), fi.fi_delta_args(**{**ok, **kw}))
    ran = fi.FI_OK if b == 0 else NO_DEVICE
    check(call("prompt"), ran, ok)
    check(call("step", lens=0, L=1), ran, ok)
    check(call("prompt", state=0, fresh=1), ran, ok)
    for kw in (dict(B=B + 1), dict(B=-1), dict(L=L + 1), dict(L=-1), dict(n_slots=-1), dict(n_slots=1 << 31), dict(state=P + 4),
               dict(lens=P + 2), dict(slots=P + 1), dict(state=0, fresh=0), dict(q=fi.fi_view(P + 1, 0, 0, 0)), dict(beta=fi.fi_view(P + 2, 0, 0, 0))):
        check(call("prompt", **kw), INVALID, kw)
    check(call("step", L=2), INVALID, "L")
    # heads
    d = rng.randint(1, 256)
    h2 = handle(fi.fi_rotary_config(B=B, L=L, Hq=Hk * G, Hk=rng.choice((0, Hk)), d=d, rot=rng.randint(0, d) // 2 * 2, norm=rng.randint(0, 2),
                                    pairs=rng.randint(0, 1), io_dtype=io))
    ok2 = dict(B=b, L=l, q=v(), k=v(), qo=v(), ko=v(), wq=rng.choice((0, P + 4)), wk=rng.choice((0, P)), first=rng.choice((0, P)))
    call2 = lambda **kw: lib.fi_rotary_run(ctypes.addressof(h2), fi.fi_rotary_args(**{**ok2, **kw}))
    some = b > 0 and l > 0
    check(call2(), NO_DEVICE if some else fi.FI_OK, ok2)
    for kw in (dict(B=B + 1), dict(B=-1), dict(L=L + 1), dict(L=-1)) + ((dict(q=fi.fi_view(0, 0, 0, 0)), dict(qo=fi.fi_view(P + 1, 0, 0, 0)),
               dict(first=P, positions=P), dict(positions=P + 2, first=0)) if some else ()):
        check(call2(**kw), INVALID, kw)
    # drafts
    N = rng.randint(0, 63)
    R, V = spread(1, (1 << 22) // (2 * N + 1)), spread(1, (1 << 31) - 1)
    h3 = handle(fi.fi_verify_config(B=R, N=N, V=V, io_dtype=io, scale=1.0, draft_scale=0.5))
    r, n = rng.choice((R, 1, spread(1, R), 0)), rng.randint(0, N)
    ok3 = dict(B=r, N=n, target=P, target_row=rng.choice((0, V * 7)), target_ld=rng.choice((0, V)), draft=rng.choice((0, P)), draft_row=V, draft_ld=V,
               tokens=P, lens=rng.choice((0, P)), u=P, r=P, out=P, kept=P, logprob=rng.choice((0, P)))
    call3 = lambda **kw: lib.fi_verify_run(ctypes.addressof(h3), fi.fi_verify_args(**{**ok3, **kw}))
    got = call3()
    check(got, fi.FI_OK if r == 0 else NO_DEVICE + (INVALID,), ok3)    # (the largest strides overflow)
    for kw in (dict(B=R + 1), dict(B=-1), dict(N=N + 1), dict(N=-1)) + ((dict(target=0), dict(r=0), dict(out=0), dict(kept=0), dict(target_row=-1),
               dict(target_ld=1 << 62), dict(target=P + 1), dict(out=P + 4), dict(kept=P + 2), dict(logprob=P + 1)) if r else ()):
        check(call3(**kw), INVALID, kw)
for f, x in ((lib.fi_delta_prompt, h), (lib.fi_delta_step, h), (lib.fi_rotary_run, h2), (lib.fi_verify_run, h3)):
    check(f(None, f.argtypes[1]._type_()), INVALID, f)
    check(f(ctypes.addressof(x), None), INVALID, f)
print("probe ok", calls)
'''


@pytest.mark.skipif(not Path(san.HIPCC).exists(), reason="hipcc missing")
def test_host_code_of_drafts_under_asan_ubsan(tmp_path):
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
    objs = [str(tmp_path / (src.name + ".o")) for src in fib.SOURCES]
    for p in [subprocess.Popen([fib.HIPCC, *flags, "-c", str(src), "-o", o], stderr=subprocess.DEVNULL) for src, o in zip(fib.SOURCES, objs)]:
        assert p.wait() == 0
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
