"""Elements behind the turned part of a head (fi_rotary_*): they are normed and weighted and
nothing else, so that an infinity or a NaN among them reaches no other element but by the norm.
Bounds as in tests/test_gpu_rotary.py."""
import math

import pytest

import draft_reference as ref
from fi_harness import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)
from test_gpu_rotary import DT, freqs, gen, size_of_pairs, stream  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 0), (128, 64), (80, 48), (72, 36), (33, 10), (7, 4), (256, 254), (255, 2)])
def test_what_is_not_turned_stays_by_itself(d, rot, norm, adjacent, dtype):
    g, dt, inv = gen(d + rot), DT[dtype][0], freqs(rot)
    q = torch.randn(2, 5, 4, d, generator=g).to(dt)
    q[0, :, 0, rot] = math.inf
    q[1, :, 0, d - 1] = -math.inf
    q[0, ::2, 1, (rot + d) // 2] = math.nan
    q[1, 3, 2, rot:] = math.inf          # all of them; head 3 has none
    w = (1.0 + 0.3 * torch.randn(d, generator=g)).to(dt)
    first = torch.tensor([0, 1000], dtype=torch.int32)
    where = torch.arange(5)[None] + first[:, None]
    out = torch.full((2, 5, 4, d), 5.0, dtype=dt, device="cuda")
    log("case rotary rest", d, rot, "norm", norm, "adjacent", adjacent, dtype)
    with fi.Rotary(2, 5, 4, 0, d, inv.cuda(), norm, 1e-6, fi.FI_PAIRS_ADJACENT if adjacent else fi.FI_PAIRS_HALVES, DT[dtype][1], stream()) as op:
        op.run(q.cuda(), None, out, None, wq=w.cuda(), first=first.cuda())
        torch.cuda.synchronize()
    got, want = out.cpu().double(), ref.rotary(q, w, where, inv, norm, 1e-6, adjacent)
    some = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    pair = size_of_pairs(q, w, inv, norm, 1e-6, adjacent)
    bound = 1e-6 * pair + (2.0 ** -8 * (want.abs() + 1e-6 * pair) if dtype == "bf16" else 2.0 ** -24 * want.abs())
    assert bool(((got - want).abs() <= bound + 1e-38)[some].all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 32), (33, 10), (128, 0)])
def test_the_rest_of_a_plain_head_keeps_its_bits(d, rot, adjacent, dtype):
    """Without a norm and weights it is copied: signs of zeros too."""
    q = torch.randn(1, 4, 3, d, generator=gen(rot)).to(DT[dtype][0])
    q[..., rot::3] = -0.0
    out = torch.empty_like(q, device="cuda")
    with fi.Rotary(1, 4, 3, 0, d, freqs(rot).cuda(), fi.FI_NORM_NONE, 0.0, fi.FI_PAIRS_ADJACENT if adjacent else fi.FI_PAIRS_HALVES, DT[dtype][1],
                   stream()) as op:
        op.run(q.cuda(), None, out, None)
        torch.cuda.synchronize()
    bits = {"bf16": torch.int16, "f32": torch.int32}[dtype]
    assert torch.equal(out[..., rot:].cpu().view(bits), q[..., rot:].contiguous().view(bits))
