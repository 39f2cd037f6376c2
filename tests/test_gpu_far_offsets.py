"""Views whose offsets pass 32 bits: rows and positions far apart in large buffers, against the
same numbers close together.  Values do not depend on strides, so they are equal where the
same route takes them, and within the operators' bounds otherwise."""
import pytest

import draft_reference as ref
from fi_harness import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)


def stream():
    return torch.cuda.current_stream()


def spread(x, strides, buf):
    """x [...] copied into buf at these strides (the last one 1)."""
    y = buf.as_strided(x.shape, strides)
    y.copy_(x)
    return y


@pytest.mark.parametrize("L", [1, 12, 70])
@pytest.mark.parametrize("far", ["rows", "positions"])
def test_delta(far, L):
    if far == "positions" and L == 1:
        pytest.skip("a single position")
    B, Hk, Hv, d = 2, 2, 2, 64
    g = torch.Generator().manual_seed(L)
    q, k = (torch.nn.functional.normalize(torch.randn(B, L, Hk, d, generator=g), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn(B, L, Hv, d, generator=g).bfloat16()
    ld, beta = -torch.rand(B, L, Hv, generator=g), torch.rand(B, L, Hv, generator=g)
    st = torch.randn(B, Hv, d, d, generator=g)
    ro, rs = ref.delta(q, k, v, ld, beta, 1.0, st)
    pos = 4 * Hk * d if far == "rows" else (1 << 32) // L // 64 * 64 + 64
    row = (1 << 31) + 64 if far == "rows" else 2 * Hk * d * 2
    buf = torch.empty((B - 1) * row + L * pos + 4 * Hk * d, dtype=torch.bfloat16, device="cuda")
    log("case far delta", far, L, "elements", buf.numel())
    n = Hk * d
    dq, dk, dv_, do = (spread(x.cuda(), (row, pos, d, 1), buf[i * n:]) for i, x in enumerate((q, k, v, torch.zeros_like(v))))
    gate = torch.empty((B - 1) * (1 << 31) + L * 2 * Hv, device="cuda") if far == "rows" else torch.empty(B * L * 2 * Hv, device="cuda")
    gs = ((1 << 31) if far == "rows" else L * 2 * Hv, 2 * Hv, 1)
    dl, db = spread(ld.cuda(), gs, gate), spread(beta.cuda(), gs, gate[Hv:])
    state = st.cuda()
    with fi.DeltaRule(B, L, Hk, Hv, d, d, 1.0, fi.FI_BF16, stream()) as op:
        op.prompt(dq, dk, dv_, dl, db, do, state)
        torch.cuda.synchronize()
    o = do.cpu().double()
    assert bool(((o - ro).abs() <= 2.0 ** -8 * ro.abs() + 2.0 ** -11 * ro.abs().max()).all())
    assert float((state.cpu().double() - rs).norm() / rs.norm()) <= 1e-5


def test_rotary():
    B, L, H, d = 2, 3, 2, 64
    x = torch.randn(B, L, H, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    freq = torch.tensor([1e4 ** (-i / 32) for i in range(32)]).cuda()
    near = x.cuda()
    want = torch.empty_like(near)
    row = (1 << 31) + 128
    buf = torch.empty(row + L * H * d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(buf)
    log("case far rotary", buf.numel())
    with fi.Rotary(B, L, H, 0, d, freq, stream=stream()) as op:
        op.run(near, None, want, None)
        y = out.as_strided(x.shape, (row, H * d, d, 1))
        op.run(spread(near, (row, H * d, d, 1), buf), None, y, None)
        torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("far", ["rows", "places"])
def test_verify(far):
    B, N, V = 2, 2, 5000
    g = torch.Generator().manual_seed(2)
    t, d = (torch.randn(B, n, V, generator=g).mul(3).bfloat16() for n in (N + 1, N))
    x = torch.randint(V, (B, N), generator=g)
    u, r = torch.rand(B, N, generator=g) * 0.1, torch.rand(B, generator=g)
    want = ref.verify(t, d, x, None, u, r)
    strides = ((1 << 31) + 8, V, 1) if far == "rows" else (V, (1 << 31) + 8, 1)
    buf = torch.empty(2 * ((1 << 31) + 8) + 3 * V, dtype=torch.bfloat16, device="cuda")
    buf2 = torch.empty_like(buf)
    out, kept = torch.empty(B, N + 1, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    log("case far verify", far, buf.numel())
    with fi.DraftCheck(B, N, V, fi.FI_BF16, stream=stream()) as op:
        op.run(spread(t.cuda(), strides, buf), x.cuda(), u.cuda(), r.cuda(), out, kept, draft=spread(d.cuda(), strides, buf2))
        torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
