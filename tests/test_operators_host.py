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
