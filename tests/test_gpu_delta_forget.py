"""The delta rule where states are forgotten: a decay far below one leaves a a S, to fp32's digits, however large S was
before, in every form.  Bounds: the state's of tests/test_gpu_delta.py, 1e-5 of the norm of what is left.  Of a decay e^G, 1.1e-7 |G| of
itself among it: G is held to 2^-48, G log2(e) rounded three times (2^-24, 2^-24, 2^-25) on its way to a power of two, which is
off by 2^-23."""
import math

import pytest

import draft_reference as ref
from fi_harness import log
from op_reference import rel_l2

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)
from test_gpu_delta import DT, TOL, TOL_STATE, inputs, stream  # noqa: E402

# steps, chunks of 16 in one launch, whole chunks, segments
LENGTHS = {"bf16": [2, 20, 100, 1300], "f32": [4, 20, 100, 700]}
FORMS = [(d, L, "prompt") for d in LENGTHS for L in LENGTHS[d]] + [(d, 3, "step") for d in LENGTHS]


def run(x, dtype, mode):
    q, k, v, ld, beta, state = x
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    ro, rs = ref.delta(*x[:5], 1.0, state)
    d, st = [y.cuda() for y in x[:5]], state.cuda()
    o = torch.full((B, L, Hv, dv), 7.0, dtype=q.dtype, device="cuda")
    log("case forget", mode, dtype, "L", L, "d", dk, dv)
    with fi.DeltaRule(B, L, Hk, Hv, dk, dv, 1.0, DT[dtype][1], stream()) as op:
        if mode == "prompt":
            op.prompt(*d, o, st)
        else:
            for t in range(L):
                op.step(*(y[:, t:t + 1] for y in d), o[:, t:t + 1], st)
        torch.cuda.synchronize()
    return o.cpu().double(), st.cpu().double(), ro, rs


@pytest.mark.parametrize("dtype,L,mode", FORMS)
@pytest.mark.parametrize("gate", [-8.0, -16.0, -30.0])
def test_a_large_state_is_forgotten(gate, dtype, L, mode):
    """States 10^4 times what the values write, one strong gate at the last position but one."""
    x = list(inputs(L, 1, L, 2, 2, 64, 48, dtype, memory=(1e3, 1e5)))
    x[5] = x[5] * 1e4
    x[3][:, L - 2] = gate
    o, st, ro, rs = run(x, dtype, mode)
    for n in range(2):
        assert rel_l2(st[0, n], rs[0, n]) <= TOL_STATE, (n, rel_l2(st[0, n], rs[0, n]))
        assert rel_l2(o[0, L - 2:, n], ro[0, L - 2:, n]) <= TOL[dtype]


@pytest.mark.parametrize("dtype,L,mode", FORMS)
@pytest.mark.parametrize("whole", [-0.2, -0.69, -0.7, -3.0, -20.0, -50.0])
def test_nothing_but_decays(whole, dtype, L, mode):
    """beta = 0: S e^G, and G is `whole` over all positions."""
    x = list(inputs(L + 1, 1, L, 2, 2, 64, 48, dtype))
    x[4][:] = 0.0
    x[3] = x[3] * (whole / x[3].double().sum(1, keepdim=True)).float()
    _, st, _, rs = run(x, dtype, mode)
    for n in range(2):
        assert rel_l2(st[0, n], rs[0, n]) <= TOL_STATE, (n, rel_l2(st[0, n], rs[0, n]))
    assert math.isclose(float(rs.norm() / x[5].double().norm()), math.exp(whole), rel_tol=1e-3)
