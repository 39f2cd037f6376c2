"""CPU checks of the delta rule, the normed and turned heads and the check of drafts
(fi_delta_*, fi_rotary_*, fi_verify_*): structures have the header's layout, create
calls and calls on a handle refuse bad arguments before any device work, the
binding checks its tensors.  A handle is made of host memory here, with
the layout of its structure, as a create call needs a device."""
import ctypes
import os
import subprocess

import pytest

import exact_online_amd as fi

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("fi_delta_config", "fi_delta_args", "fi_rotary_config", "fi_rotary_args", "fi_verify_config", "fi_verify_args")
INF, NAN = float("inf"), float("nan")
P = 4096   # a stand-in device pointer: nothing is launched


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
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fi.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True, capture_output=True)
    assert [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want
    assert fi._DELTA_ARGS.size == ctypes.sizeof(fi.fi_delta_args) and fi._ROTARY_ARGS.size == ctypes.sizeof(fi.fi_rotary_args)


DELTA = dict(B=2, L=16, Hk=2, Hv=4, dk=8, dv=8, scale=1.0, io_dtype=0)
ROTARY = dict(B=2, L=16, Hq=4, Hk=2, d=8, rot=8, norm=1, eps=1e-6, pairs=0, io_dtype=0)
VERIFY = dict(B=2, N=3, V=100, io_dtype=0, scale=1.0, draft_scale=1.0)
KINDS = {"delta": (fi.fi_delta_config, DELTA), "rotary": (fi.fi_rotary_config, ROTARY), "verify": (fi.fi_verify_config, VERIFY)}


def create(kind, **kw):
    C, base = KINDS[kind]
    out = ctypes.c_void_p(123)
    args = (ctypes.byref(C(**{**base, **kw})),) + ((P,) if kind == "rotary" else ())
    return getattr(fi.lib, f"fi_{kind}_create")(*args, ctypes.byref(out)), out.value


BIG = (1 << 31, 1 << 40, (1 << 63) - 1, -(1 << 63))


@pytest.mark.parametrize("kind,kw", [
    *[("delta", {n: v}) for n in ("B", "L", "Hk", "Hv", "dk", "dv") for v in (0, -1, -(1 << 63))],
    *[("delta", {n: v}) for n in ("B", "L") for v in BIG],
    ("delta", dict(Hk=3)), ("delta", dict(Hk=8)), ("delta", dict(scale=INF)), ("delta", dict(scale=NAN)), ("delta", dict(io_dtype=2)),
    ("delta", dict(io_dtype=-1)), ("delta", dict(B=1 << 20, L=1 << 20, Hv=1 << 10)),
    *[("rotary", {n: v}) for n in ("B", "L", "Hq", "d") for v in (0, -1)], ("rotary", dict(Hk=-1)), ("rotary", dict(rot=-2)),
    ("rotary", dict(rot=3)), ("rotary", dict(rot=10)), ("rotary", dict(norm=3)), ("rotary", dict(norm=-1)), ("rotary", dict(pairs=2)),
    ("rotary", dict(eps=-1.0)), ("rotary", dict(eps=NAN)), ("rotary", dict(eps=INF)), ("rotary", dict(io_dtype=2)),
    ("rotary", dict(B=1 << 20, L=1 << 30)), *[("rotary", {n: v}) for n in ("B", "L", "Hq", "Hk") for v in BIG],
    *[("verify", {n: v}) for n in ("B", "V") for v in (0, -1, *BIG)], ("verify", dict(N=-1)), ("verify", dict(N=64)), ("verify", dict(io_dtype=2)),
    *[("verify", {n: v}) for n in ("scale", "draft_scale") for v in (0.0, -1.0, NAN, INF)],
])
def test_create_refuses(kind, kw):
    assert create(kind, **kw) == (fi.FI_ERR_INVALID, None)


@pytest.mark.parametrize("kind,kw", [("delta", dict(dk=257)), ("delta", dict(dv=1000)), ("delta", dict(L=fi.FI_MAX_L + 1)),
                                     ("delta", dict(B=1 << 20, Hk=1, Hv=2)), ("rotary", dict(d=258)), ("verify", dict(B=1 << 21, N=1))])
def test_create_unsupported_sizes(kind, kw):
    assert create(kind, **kw) == (fi.FI_ERR_UNSUPPORTED, None)


def test_null_arguments():
    for kind, (C, base) in KINDS.items():
        fn = getattr(fi.lib, f"fi_{kind}_create")
        dev = (P,) if kind == "rotary" else ()
        out = ctypes.c_void_p(123)
        assert fn(None, *dev, ctypes.byref(out)) == fi.FI_ERR_INVALID and out.value is None
        assert fn(ctypes.byref(C(**base)), *dev, None) == fi.FI_ERR_INVALID
        getattr(fi.lib, f"fi_{kind}_destroy")(None)
    out = ctypes.c_void_p(123)
    assert fi.lib.fi_rotary_create(ctypes.byref(fi.fi_rotary_config(**ROTARY)), None, ctypes.byref(out)) == fi.FI_ERR_INVALID
    for fn in (fi.lib.fi_delta_prompt, fi.lib.fi_delta_step, fi.lib.fi_rotary_run, fi.lib.fi_verify_run):
        assert fn(None, fn.argtypes[1]._type_()) == fi.FI_ERR_INVALID


def test_create_without_gpu_is_unsupported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for kind in KINDS:
        assert create(kind) == (fi.FI_ERR_UNSUPPORTED, None)


# ------------------------------------------------------------ calls on a handle
def handle(cfg):
    class H(ctypes.Structure):
        _fields_ = [("cfg", type(cfg)), ("stream", ctypes.c_void_p), ("device", ctypes.c_int), ("p", ctypes.c_void_p * 4)]
    return H(cfg, None, 0, (ctypes.c_void_p * 4)(P, P, P, P))


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the handles are not of this device")


@no_gpu
def test_delta_calls():
    h = handle(fi.fi_delta_config(**DELTA))
    v, g = fi.fi_view(P, 512, 32, 8), fi.fi_view(P, 64, 4, 1)
    ok = dict(B=2, L=16, q=v, k=v, v=v, o=v, log_decay=g, beta=g, n_slots=2, state=P)

    def call(name, **kw):
        return getattr(fi.lib, f"fi_delta_{name}")(ctypes.addressof(h), fi.fi_delta_args(**{**ok, **kw}))
    assert call("prompt") == fi.FI_ERR_HIP          # it would launch
    assert call("prompt", B=0) == fi.FI_OK
    assert call("step", L=1) == fi.FI_ERR_HIP
    assert call("prompt", state=0, n_slots=0, fresh=1) == fi.FI_ERR_HIP
    odd = fi.fi_view(P + 2, 0, 0, 0)
    for kw in (dict(B=3), dict(B=-1), dict(L=17), dict(L=-1), dict(n_slots=1), dict(n_slots=-1), dict(n_slots=1 << 31), dict(state=0),
               dict(state=P + 4), dict(lens=P + 2), dict(slots=P + 1), *({n: fi.fi_view(0, 0, 0, 0)} for n in ("q", "k", "v", "o", "log_decay", "beta")),
               *({n: odd} for n in ("q", "k", "v", "o", "log_decay", "beta"))):
        assert call("prompt", **kw) == fi.FI_ERR_INVALID, kw
    for kw in (dict(L=2), dict(L=1, lens=P), dict(L=0), dict(L=1, state=0, fresh=1, n_slots=0)):
        assert call("step", **kw) == fi.FI_ERR_INVALID, kw
    assert fi.lib.fi_delta_prompt(ctypes.addressof(h), None) == fi.FI_ERR_INVALID


@no_gpu
def test_rotary_calls():
    h = handle(fi.fi_rotary_config(**ROTARY))
    v = fi.fi_view(P, 512, 32, 8)
    ok = dict(B=2, L=16, q=v, k=v, qo=v, ko=v)

    def call(**kw):
        return fi.lib.fi_rotary_run(ctypes.addressof(h), fi.fi_rotary_args(**{**ok, **kw}))
    assert call() == fi.FI_ERR_HIP and call(B=0, q=fi.fi_view()) == fi.FI_OK and call(L=0) == fi.FI_OK
    for kw in (dict(B=3), dict(B=-1), dict(L=17), dict(L=-1), *({n: fi.fi_view(0, 0, 0, 0)} for n in ("q", "k", "qo", "ko")),
               *({n: fi.fi_view(P + 1, 0, 0, 0)} for n in ("q", "k", "qo", "ko")), dict(first=P, positions=P), dict(first=P + 2),
               dict(positions=P + 1), dict(wq=P + 2), dict(wk=P + 1)):
        assert call(**kw) == fi.FI_ERR_INVALID, kw
    h2 = handle(fi.fi_rotary_config(**{**ROTARY, "Hk": 0}))
    assert fi.lib.fi_rotary_run(ctypes.addressof(h2), fi.fi_rotary_args(**{**ok, "k": fi.fi_view(), "ko": fi.fi_view()})) == fi.FI_ERR_HIP
    assert fi.lib.fi_rotary_run(ctypes.addressof(h), None) == fi.FI_ERR_INVALID


@no_gpu
def test_verify_calls():
    h = handle(fi.fi_verify_config(**VERIFY))
    ok = dict(B=2, N=3, target=P, target_row=400, target_ld=100, draft=P, draft_row=300, draft_ld=100, tokens=P, lens=P, u=P, r=P, out=P,
              kept=P, logprob=P)

    def call(**kw):
        return fi.lib.fi_verify_run(ctypes.addressof(h), fi.fi_verify_args(**{**ok, **kw}))
    assert call() == fi.FI_ERR_HIP and call(B=0, target=0) == fi.FI_OK
    assert call(draft=0, lens=0, logprob=0) == fi.FI_ERR_HIP and call(N=0, tokens=0, u=0) == fi.FI_ERR_HIP
    for kw in (dict(B=3), dict(B=-1), dict(N=4), dict(N=-1), *({n: 0} for n in ("target", "tokens", "u", "r", "out", "kept")),
               *({n: -1} for n in ("target_row", "target_ld", "draft_row", "draft_ld")), *({n: 1 << 62} for n in ("target_row", "draft_ld")),
               *({n: P + 2} for n in ("target", "draft", "lens", "u", "r", "kept", "logprob")), *({n: P + 4} for n in ("tokens", "out"))):
        assert call(**kw) == fi.FI_ERR_INVALID, kw
    assert fi.lib.fi_verify_run(ctypes.addressof(h), None) == fi.FI_ERR_INVALID


# ------------------------------------------------------------ the binding
class OnDevice:
    """A tensor that says it lies on device 0."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


class Calls:
    """Stands in for the library: says FI_OK and counts the calls that run something."""

    def __init__(self):
        self.n = 0

    def __getattr__(self, name):
        def call(*a):
            if name == "fi_strerror":
                return b""
            if name.endswith("_create"):
                a[-1]._obj.value = 1
            elif not name.endswith("_destroy"):
                self.n += 1
                self.args = a[-1]
            return fi.FI_OK
        return call


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(fi, "lib", c)
    return c


def zeros(*shape, t=torch.float32):
    return torch.zeros(*shape, dtype=t)


BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
OTHER = {BF: F32, F32: BF, I32: I64, I64: I32}


def check_binding(calls, op, ok, any_stride):
    """Every tensor of another type, too short, on the host, and with gaps in its last dimension."""
    dev = {n: OnDevice(t) for n, t in ok.items()}
    n = calls.n
    op(**dev)
    assert calls.n == n + 1
    for name, t in ok.items():
        bad = [OnDevice(t.to(OTHER[t.dtype])), OnDevice(t[..., :-1].contiguous()), t]
        if name not in any_stride:
            bad.append(OnDevice(zeros(*t.shape[:-1], 2 * t.shape[-1], t=t.dtype)[..., ::2]))
        for x in bad:
            with pytest.raises(fi.FiError) as e:
                op(**{**dev, name: x})
            assert e.value.status == fi.FI_ERR_INVALID, name
            assert calls.n == n + 1, name


@no_gpu
def test_delta_rule_checks_its_tensors(calls):
    ok = dict(q=zeros(3, 4, 2, 8, t=BF), k=zeros(3, 4, 2, 8, t=BF), v=zeros(3, 4, 4, 6, t=BF), log_decay=zeros(3, 4, 4), beta=zeros(3, 4, 4),
              o=zeros(3, 4, 4, 6, t=BF), state=zeros(5, 4, 8, 6), lens=zeros(3, t=I32), slots=zeros(3, t=I32))
    with fi.DeltaRule(3, 4, 2, 4, 8, 6, 1.0, fi.FI_BF16) as op:
        check_binding(calls, op.prompt, ok, ("log_decay", "beta"))
        a = [OnDevice(ok[n]) for n in ("q", "k", "v", "log_decay", "beta", "o")]
        op.prompt(*a, fresh=True, hold=True)
        assert (calls.args.fresh, calls.args.hold, calls.args.n_slots, calls.args.state) == (1, 1, 0, None)
        op.prompt(*a, OnDevice(ok["state"]))
        assert (calls.args.B, calls.args.L, calls.args.fresh, calls.args.hold, calls.args.n_slots) == (3, 4, 0, 0, 5)
        assert (calls.args.beta.row, calls.args.beta.pos, calls.args.beta.head, calls.args.beta.p) == (16, 4, 1, ok["beta"].data_ptr())
        for state in (zeros(5, 4, 6, 8), zeros(5, 4, 6, 8).transpose(2, 3), zeros(960), torch.tensor(0.0)):
            with pytest.raises(fi.FiError):
                op.prompt(*a, OnDevice(state))


@no_gpu
def test_rotary_checks_its_tensors(calls):
    ok = dict(q=zeros(3, 4, 4, 8, t=BF), k=zeros(3, 4, 2, 8, t=BF), qo=zeros(3, 4, 4, 8, t=BF), ko=zeros(3, 4, 2, 8, t=BF), wq=zeros(8, t=BF),
              wk=zeros(8, t=BF), first=zeros(3, t=I32))
    for bad in (zeros(4), OnDevice(zeros(4, t=BF)), OnDevice(zeros(8)[::2])):
        with pytest.raises(fi.FiError):
            fi.Rotary(3, 4, 4, 2, 8, bad)
    with fi.Rotary(3, 4, 4, 2, 8, OnDevice(zeros(4))) as op, fi.Rotary(3, 4, 4, 0, 8, None) as one:
        assert op.cfg.rot == 8 and one.cfg.rot == 0
        check_binding(calls, op.run, ok, ())
        ok.pop("first")
        check_binding(calls, op.run, ok | dict(positions=zeros(3, 4, t=I32)), ())
        one.run(OnDevice(ok["q"]), None, OnDevice(ok["qo"]), None)
        assert (calls.args.k.p, calls.args.wq, calls.args.q.head) == (None, None, 8)


@no_gpu
def test_draft_check_checks_its_tensors(calls):
    ok = dict(target=zeros(3, 5, 50, t=BF), tokens=zeros(3, 4, t=I64), u=zeros(3, 4), r=zeros(3), out=zeros(3, 5, t=I64), kept=zeros(3, t=I32),
              logprob=zeros(3, 5), draft=zeros(3, 4, 50, t=BF), lens=zeros(3, t=I32))
    with fi.DraftCheck(3, 4, 50, fi.FI_BF16) as op:
        check_binding(calls, op.run, ok, ())
        op.run(*(OnDevice(ok[n]) for n in ("target", "tokens", "u", "r", "out", "kept")))
        assert (calls.args.N, calls.args.target_row, calls.args.target_ld, calls.args.draft, calls.args.logprob) == (4, 250, 50, None, None)
