"""The largest sizes that the delta rule and the check of drafts take: FI_MAX_L positions, 2^31 - 1 tokens."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)
from fi_harness import log  # noqa: E402

DT = {"bf16": (torch.bfloat16, fi.FI_BF16), "f32": (torch.float32, fi.FI_F32)}


def stream():
    return torch.cuda.current_stream()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_longest_prompt(dtype):
    """Nothing is written to the state (beta = 0): S[t] = S[0] e^{g t}, o[t] = S[t]^T q[t].  A chunk's decay of an fp32 value is
    rounded once, by at most 2^-24 of it; with the same gate everywhere always to the same side (a chunk takes 107.4
    units of the last place from 1, and every segment begins there: 107): (1 + 2^-24)^chunks - 1 in all."""
    L, d, g = fi.FI_MAX_L, 16, -1e-7
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    dt = DT[dtype][0]
    q = torch.nn.functional.normalize(torch.randn(1, L, 1, d, generator=gen, device="cuda"), dim=-1).to(dt)
    v = torch.randn(1, L, 1, d, generator=gen, device="cuda").to(dt)
    state = torch.randn(1, 1, d, d, generator=gen, device="cuda")
    gates = torch.full((1, 1, 1), g, device="cuda").expand(1, L, 1)
    beta = torch.zeros(1, 1, 1, device="cuda").expand(1, L, 1)
    o, st = torch.full((1, L, 1, d), 7.0, dtype=dt, device="cuda"), state.clone()
    log("case longest prompt", dtype)
    with fi.DeltaRule(1, L, 1, 1, d, d, 1.0, DT[dtype][1], stream()) as op:
        op.prompt(q, q, v, gates, beta, o, st)
        torch.cuda.synchronize()
    g = float(torch.tensor(g))   # as fp32 has it
    lost = math.expm1(L / (64 if dtype == "bf16" else 32) * 2.0 ** -24) + 1e-6
    want = state.double() * math.exp(g * L)
    assert float((st.double() - want).norm() / want.norm()) <= lost
    at = torch.cat([torch.arange(0, L, 9973), torch.arange(L - 200, L)]).cuda()
    want = (q[0, at, 0].double() @ state[0, 0].double()) * torch.exp(g * (at + 1).double())[:, None]
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    size = q[0, at, 0].double().abs() @ state[0, 0].double().abs()
    assert bool(((o[0, at, 0].double() - want).abs() <= step * want.abs() + (lost + 2.0 ** -16 * (dtype == "bf16")) * size).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_vocabulary(dtype):
    """2^31 - 1 tokens, all alike: r falls on token floor(r V); with one left out, on the next from there on."""
    V = (1 << 31) - 1
    dt = DT[dtype][0]
    r = torch.tensor([0.0, 0.3, 0.75, 0.9])
    z = torch.zeros(1, 1, V, dtype=dt, device="cuda")
    z[0, 0, V - 1] = -math.inf
    n = V - 1
    places = [float(x) * n for x in r]
    assert all(x == 0.0 or 0.02 < x % 1.0 < 0.98 for x in places)   # none near a border
    out, kept = torch.empty(4, 2, dtype=torch.int64, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    lp = torch.empty(4, 2, device="cuda")
    log("case largest vocabulary", dtype)
    with fi.DraftCheck(4, 1, V, DT[dtype][1], stream=stream()) as op:
        x, u = torch.full((4, 1), 5, dtype=torch.int64, device="cuda"), torch.full((4, 1), 0.5, device="cuda")
        alone = torch.empty(4, 1, dtype=torch.int64, device="cuda")
        op.run(z.expand(4, 1, V), x[:, :0].contiguous(), u[:, :0].contiguous(), r.cuda(), alone, kept)
        torch.cuda.synchronize()
        assert alone[:, 0].tolist() == [int(x) for x in places] and kept.tolist() == [0] * 4
        op.run(z.expand(4, 2, V), x, u, r.cuda(), out, kept, lp)                    # a certain draft, not kept
        torch.cuda.synchronize()
    left = [float(y) * (n - 1) for y in r]
    assert all(y == 0.0 or 0.02 < y % 1.0 < 0.98 for y in left)
    assert out.tolist() == [[int(y) + (int(y) >= 5), -1] for y in left] and kept.tolist() == [0] * 4
    assert bool(((lp[:, 0].double().cpu() + math.log(n)).abs() <= 2.0 ** -24 * math.log(n) + 1e-11).all())
