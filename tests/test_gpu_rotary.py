"""GPU parity of normed and turned heads (fi_rotary_*) against 64 bits.

Bounds: an output is x f w cos -+ x' f w' sin, each factor off by at most 2^-23 (f: a sum of 256 squares,
8 half ulps; a quotient, a root) and cos and sin by 3e-8 of 1: 16 * 2^-24 = 1e-6 of the pair's size
for fp32, and one rounding (2^-8) more for bf16."""
import math

import pytest

import draft_reference as ref
from fi_harness import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)

DT = {"bf16": (torch.bfloat16, fi.FI_BF16), "f32": (torch.float32, fi.FI_F32)}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def stream():
    return torch.cuda.current_stream()


def freqs(rot, base=1e4):
    return torch.tensor([base ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32)


def near(got, want, pair, dtype):
    """pair: the size of what an element is made of."""
    got, want = got.cpu().double(), want.double()
    bound = 1e-6 * pair + (2.0 ** -8 * (want.abs() + 1e-6 * pair) if dtype == "bf16" else 2.0 ** -24 * want.abs())
    over = ((got - want).abs() - bound - 1e-38).max() if got.numel() else torch.tensor(-1.0)
    log("rotary max excess %.3g" % float(over))
    assert bool(torch.isfinite(got).all()) and float(over) <= 0.0


def size_of_pairs(x, w, inv, norm, eps, adjacent):
    plain = ref.rotary(x, w, torch.zeros(x.shape[:2]), inv[:0], norm, eps, adjacent).abs()
    size = plain.clone()
    for i in range(len(inv)):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + len(inv))
        size[..., a] = size[..., b] = plain[..., a] + plain[..., b]
    return size


def check(seed, B, L, Hq, Hk, d, rot, norm, adjacent, dtype, weights=True, first=None, positions=None, layout="fused", eps=1e-6):
    g, dt = gen(seed), DT[dtype][0]
    inv = freqs(rot)
    q, k = (torch.randn(B, L, h, d, generator=g).to(dt) for h in (Hq, Hk))
    wq, wk = ((1.0 + 0.3 * torch.randn(d, generator=g)).to(dt) if weights else None for _ in range(2))
    where = torch.arange(L)[None].expand(B, L)
    if first is not None:
        where = where + torch.tensor(first)[:, None]
    if positions is not None:
        where = positions
    log("case rotary", B, L, Hq, Hk, d, rot, "norm", norm, "adjacent", adjacent, dtype, layout)
    start = 1 if layout == "odd" else 0
    buf = torch.full((B, L, (Hq + Hk) * d + 3 * (layout == "odd")), 9.0, dtype=dt, device="cuda")
    buf[..., start:start + Hq * d] = q.reshape(B, L, -1).cuda()
    buf[..., start + Hq * d:start + (Hq + Hk) * d] = k.reshape(B, L, -1).cuda()
    dq = buf[..., start:start + Hq * d].unflatten(-1, (Hq, d))
    dk = buf[..., start + Hq * d:start + (Hq + Hk) * d].unflatten(-1, (Hk, d)) if Hk else None
    in_place = layout == "in_place"
    qo = dq if in_place else torch.full((B, Hq, L, d), 5.0, dtype=dt, device="cuda").transpose(1, 2)
    ko = dk if in_place else torch.full((B, L, Hk, d), 5.0, dtype=dt, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    with fi.Rotary(B, L, Hq, Hk, d, inv.cuda(), norm, eps, fi.FI_PAIRS_ADJACENT if adjacent else fi.FI_PAIRS_HALVES, DT[dtype][1],
                   stream()) as op:
        op.run(dq, dk, qo, ko, wq=None if wq is None else wq.cuda(), wk=None if wk is None else wk.cuda(),
               first=None if first is None else torch.tensor(first, **i32),
               positions=None if positions is None else positions.to(**i32).contiguous())
        torch.cuda.synchronize()
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        if x.shape[2]:
            near(y, ref.rotary(x, w, where, inv, norm, eps, adjacent), size_of_pairs(x, w, inv, norm, eps, adjacent), dtype)
    if not in_place:
        assert torch.equal(dq.cpu(), q)
    if layout == "odd":
        assert bool((buf[..., 0] == 9.0).all()) and bool((buf[..., -2:] == 9.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot", [(1, 0), (2, 2), (3, 2), (7, 4), (16, 16), (33, 10), (64, 64), (72, 36), (80, 48), (96, 32), (100, 100),
                                   (128, 128), (130, 64), (192, 64), (255, 254), (256, 256), (256, 0), (254, 2)])
def test_head_sizes(d, rot, adjacent, dtype):
    check(d + rot, 2, 5, 3, 2, d, rot, (d + rot) % 3, adjacent, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("layout", ["fused", "odd", "in_place"])
def test_layouts_and_norms(layout, norm, dtype):
    check(norm, 3, 40, 4, 2, 64, 32, norm, False, dtype, layout=layout, weights=norm != 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,Hq,Hk", [(1, 1, 1, 0), (1, 1, 1, 1), (1, 3000, 2, 1), (300, 1, 28, 4), (2, 700, 40, 8), (7, 1, 16, 16), (1, 9000, 1, 1)])
def test_counts(B, L, Hq, Hk, dtype):
    check(B + L, B, L, Hq, Hk, 128, 128, 1, False, dtype)


@pytest.mark.parametrize("adjacent", [False, True])
def test_far_positions(adjacent):
    """Positions to the end of 32 bits, negative ones: the angles are as good as near ones'."""
    check(1, 4, 9, 2, 2, 64, 64, 1, adjacent, "f32", first=[0, 1 << 20, (1 << 31) - 9, -(1 << 31)])
    g = gen(2)
    check(2, 2, 33, 2, 2, 64, 64, 1, adjacent, "f32", positions=torch.randint(-(1 << 31), (1 << 31) - 1, (2, 33), generator=g))


def test_small_and_empty_heads():
    """A head of zeros stays zero where eps is not; tiny heads keep what eps leaves them."""
    q = torch.zeros(1, 2, 3, 64, device="cuda")
    q[0, 1, 1] = 1e-4
    out = torch.empty_like(q)
    with fi.Rotary(1, 2, 3, 0, 64, freqs(64).cuda(), fi.FI_NORM_L2, 1e-6, fi.FI_PAIRS_HALVES, fi.FI_F32, stream()) as op:
        op.run(q, None, out, None)
        torch.cuda.synchronize()
    want = ref.rotary(q.cpu(), None, torch.arange(2)[None], freqs(64), 2, float(torch.tensor(1e-6, dtype=torch.float32)), False)
    assert float((out.cpu().double() - want).abs().max()) <= 1e-6
    assert float(out[0, 0].abs().max()) == 0.0


def test_replays_of_a_graph():
    g0 = gen(3)
    q, k = (torch.randn(2, 30, h, 64, generator=g0).bfloat16().cuda() for h in (4, 2))
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with fi.Rotary(2, 30, 4, 2, 64, freqs(64).cuda(), stream=s) as op, torch.cuda.stream(s):
        op.run(q, k, qo, ko, first=first)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            op.run(q, k, qo, ko, first=first)
        for i in range(3):
            first.fill_(1000 * i)
            g.replay()
            s.synchronize()
            a, b = qo.clone(), ko.clone()
            op.run(q, k, qo, ko, first=first)
            s.synchronize()
            assert torch.equal(a, qo) and torch.equal(b, ko)
    torch.cuda.synchronize()


def test_refusals():
    with pytest.raises(fi.FiError) as e:
        fi.Rotary(1, 1, 1, 1, 8, torch.tensor([1.0, math.inf], device="cuda"))
    assert e.value.status == fi.FI_ERR_INVALID
    q = torch.zeros(2, 4, 2, 8, device="cuda")
    i = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with fi.Rotary(2, 4, 2, 2, 8, freqs(8).cuda(), io_dtype=fi.FI_F32, stream=stream()) as op:
        def refused(*a, **kw):
            with pytest.raises(fi.FiError) as e:
                op.run(*a, **kw)
            assert e.value.status == fi.FI_ERR_INVALID
        refused(q, q[:, :3], q, q)
        refused(q, q, q.bfloat16(), q)
        refused(q, q, q, q, first=i[:, 0].contiguous(), positions=i)
        refused(q, q, q, q, positions=i[:1])
        refused(q, q, q, q, wq=torch.zeros(7, device="cuda"))
        refused(q, q, q, q.cpu())
        big = torch.zeros(2, 5, 2, 8, device="cuda")
        refused(big, big, big, big)
        op.run(q[:0], q[:0], q[:0], q[:0])
        op.run(q[:, :0], q[:, :0], q[:, :0], q[:, :0])
        op.run(q, q, q, q, positions=i)
        torch.cuda.synchronize()
