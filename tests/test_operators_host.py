"""CPU checks of the operators' calls on a handle.  A handle is made
of host memory here, with the layout of its structure, as a create call needs a
device: a call that refuses its arguments does so before it looks at one,
and a call that would launch gets an error from the runtime instead."""
import ctypes

import pytest

import exact_online_amd as fi

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("the handles are not of this device", allow_module_level=True)

P = 4096   # a stand-in device pointer: nothing is launched


class lattn_handle(ctypes.Structure):
    _fields_ = [("cfg", fi.fi_lattn_config), ("stream", ctypes.c_void_p), ("ld", ctypes.c_void_p), ("ws", ctypes.c_void_p)]


@pytest.fixture
def lattn():
    h = lattn_handle(fi.fi_lattn_config(B=2, L=16, H=4, Hkv=2, dk=8, dv=8, scale=1.0, io_dtype=fi.FI_F32), None, P, P)

    def call(name, **kw):
        view = fi.fi_view(P, 512, 32, 8)
        a = dict(B=2, L=16, q=view, k=view, v=view, o=view, n_slots=2, state=P)
        return getattr(fi.lib, f"fi_lattn_{name}")(ctypes.addressof(h), fi.fi_lattn_args(**{**a, **kw}))
    return call


@pytest.mark.parametrize("fresh", [0, 1])
@pytest.mark.parametrize("slots", [0, P])
def test_step_needs_states(lattn, fresh, slots):
    """Every step leaves a state behind: without an array for it there is nowhere to
    write, whatever it begins from.  A fresh prompt may go without."""
    kw = dict(L=1, state=0, n_slots=0, fresh=fresh, slots=slots)
    assert lattn("step", **kw) == fi.FI_ERR_INVALID
    want = fi.FI_ERR_HIP if fresh else fi.FI_ERR_INVALID
    assert lattn("prompt", **kw) == want
    assert lattn("step", **{**kw, "B": 0, "fresh": 1}) == fi.FI_OK      # no rows, no states
    assert lattn("step", L=1, fresh=fresh) == fi.FI_ERR_HIP             # with states it would launch


# ------------------------------------------------------------ the binding
class OnDevice:
    """A tensor that says it lies on the device."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

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
LATTN_OK = dict(q=zeros(3, 4, 4, 8, t=BF), k=zeros(3, 4, 2, 8, t=BF), v=zeros(3, 4, 2, 6, t=BF), o=zeros(3, 4, 4, 6, t=BF),
                state=zeros(5, 2, 8, 6), lens=zeros(3, t=I32), slots=zeros(3, t=I32))
DENSE_OK = dict(x=zeros(3, 8, t=BF), w=zeros(6, 8, t=BF), y=zeros(3, 6), bias=zeros(6, t=BF), res=zeros(3, 6))
SCORES_OK = dict(logits=zeros(3, 50, t=BF), targets=zeros(3, t=I64), logprob=zeros(3), entropy=zeros(3), lse=zeros(3),
                 top=zeros(3, 4), top_id=zeros(3, 4, t=I64))


def wrong(ok, strided):
    """(name, tensor): of another type each, too short, on the host, and (`strided`: dense arrays) with gaps."""
    for name, t in ok.items():
        other = {BF: F32, F32: BF, I32: I64, I64: I32}[t.dtype]
        yield name, OnDevice(t.to(other))
        yield name, OnDevice(t[..., :-1].contiguous())
        yield name, t
        if name in strided:
            wide = zeros(*t.shape[:-1], 2 * t.shape[-1], t=t.dtype)
            yield name, OnDevice(wide[..., ::2])


def check_binding(calls, op, ok, strided):
    ok = {n: OnDevice(t) for n, t in ok.items()}
    n = calls.n
    op(**ok)
    assert calls.n == n + 1
    for name, bad in wrong({n: t.t for n, t in ok.items()}, strided):
        with pytest.raises(fi.FiError) as e:
            op(**{**ok, name: bad})
        assert e.value.status == fi.FI_ERR_INVALID, name
        assert calls.n == n + 1, (name, bad.dtype, bad.shape)


def test_linear_attention_checks_its_tensors(calls):
    for bad in (zeros(2), OnDevice(zeros(1)), OnDevice(zeros(2, t=BF)), OnDevice(zeros(4)[::2])):
        with pytest.raises(fi.FiError):
            fi.LinearAttention(3, 4, 4, 2, 8, 6, bad, 1.0, fi.FI_BF16).close()
    with fi.LinearAttention(3, 4, 4, 2, 8, 6, OnDevice(zeros(2)), 1.0, fi.FI_BF16) as op:
        check_binding(calls, op.prompt, LATTN_OK, ("q", "k", "v", "o", "state", "lens", "slots"))
        op.prompt(**{n: OnDevice(LATTN_OK[n]) for n in "qkvo"}, fresh=True)
        for state in (zeros(5, 2, 6, 8), zeros(5, 2, 8, 5), zeros(5, 96), zeros(5, 2, 6, 8).transpose(2, 3), zeros(96),
                      zeros(5, 4, 8, 6)[:, ::2], zeros(1, 2, 8, 6).expand(5, -1, -1, -1), torch.tensor(0.0)):
            n = calls.n
            with pytest.raises(fi.FiError):
                op.step(*(OnDevice(LATTN_OK[x][:, :1]) for x in "qkvo"), state=OnDevice(state))
            assert calls.n == n


def test_dense_checks_its_tensors(calls):
    with fi.Dense(3, 6, 8, fi.FI_BF16, fi.FI_F32) as op:
        check_binding(calls, op.run, DENSE_OK, ("x", "w", "y", "res", "bias"))
        op.run(*(OnDevice(DENSE_OK[n]) for n in "xwy"))


def test_token_scores_checks_its_tensors(calls):
    with fi.TokenScores(3, 50, 4, fi.FI_BF16) as op:
        check_binding(calls, op.run, SCORES_OK, ("logits", "targets", "logprob", "entropy", "lse", "top", "top_id"))
        op.run(OnDevice(SCORES_OK["logits"]), top=OnDevice(zeros(12)), top_id=OnDevice(zeros(20, t=I64)))   # as long or longer


def test_addresses_are_taken_as_they_are(calls):
    with fi.Dense(3, 6, 8, fi.FI_BF16, fi.FI_F32) as op, fi.TokenScores(3, 50, 0, fi.FI_BF16) as sc:
        op.run(*(OnDevice(DENSE_OK[n]) for n in "xwy"), bias=P)
        sc.run(OnDevice(SCORES_OK["logits"]), targets=P, logprob=P, entropy=P)
    assert calls.n == 2


def test_the_stride_of_a_single_row_says_nothing(calls):
    """torch gives a dimension of size one any stride (a transposed column: 1), and the
    library wants rows at least their length apart."""
    def row(n, t):
        return OnDevice(zeros(n, 1, t=t).T)
    with fi.Dense(4, 6, 8, fi.FI_BF16, fi.FI_F32) as op, fi.Dense(4, 1, 8, fi.FI_BF16, fi.FI_F32) as one, \
            fi.TokenScores(4, 50, 0, fi.FI_BF16) as sc:
        op.run(row(8, BF), OnDevice(zeros(6, 8, t=BF)), row(6, F32), res=row(6, F32))
        a = calls.args
        assert (a.M, a.ldx, a.ldw, a.ldr, a.ldy) == (1, 8, 8, 6, 6)
        one.run(OnDevice(zeros(3, 8, t=BF)), row(8, BF), OnDevice(zeros(3, 1)))
        assert (calls.args.ldx, calls.args.ldw, calls.args.ldy) == (8, 8, 1)
        sc.run(row(50, BF), entropy=OnDevice(zeros(1)))
        assert (calls.args.rows, calls.args.ld) == (1, 50)
        op.run(OnDevice(zeros(2, 9, t=BF)[:, 1:]), OnDevice(zeros(6, 12, t=BF)[:, :8]), OnDevice(zeros(2, 7)[:, 1:]))
        assert (calls.args.ldx, calls.args.ldw, calls.args.ldy) == (9, 12, 7)      # of several rows it does
