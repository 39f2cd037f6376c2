"""GPU parity of the check of drafted tokens (fi_verify_*) with the same rules in 64 bits on the CPU.

Tokens and counts have to be equal.  Both sides hold probabilities to 2^-40 at least, so that a
random number falls on another token with a probability of V 2^-39 at most: 4e-7 for the
largest V here, for each row.  Log probabilities are rounded to fp32 once from 64 bits:
2^-24 of themselves, and 1e-11 that 64 bits lose."""
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


def inputs(seed, B, N, V, dtype, near=0.5, masked=0.0):
    g, dt = gen(seed), DT[dtype][0]
    base = torch.randn(B, N + 1, V, generator=g) * 3.0
    target = base.to(dt)
    draft = (base[:, :N] + near * torch.randn(B, N, V, generator=g)).to(dt)
    if masked:
        out = torch.rand(B, N + 1, V, generator=g) < masked
        out[..., 0] = False
        target.masked_fill_(out, -math.inf)
        draft.masked_fill_(out[:, :N], -math.inf)
    tokens = torch.distributions.Categorical(logits=draft.float()).sample() if N else torch.zeros(B, 0, dtype=torch.int64)
    return target, draft, tokens, torch.rand(B, N, generator=g), torch.rand(B, generator=g)


def check(x, dtype, draft=True, lens=None, pad=0, shift=0, scale=1.0, draft_scale=None, handle=None):
    target, dr, tokens, u, r = x
    B, N = tokens.shape
    V = target.shape[2]
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).item()  # noqa: E731
    want = ref.verify(target, dr if draft else None, tokens, lens, u, r, f32(scale), f32(scale if draft_scale is None else draft_scale))

    def dev(a):
        buf = torch.full((*a.shape[:2], V + pad + shift), float("nan"), dtype=a.dtype, device="cuda")
        y = buf[..., shift:shift + V]
        y.copy_(a)
        return y
    out = torch.full((B, N + 1), 77, dtype=torch.int64, device="cuda")
    kept = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    lp = torch.full((B, N + 1), 77.0, device="cuda")
    log("case verify", B, N, V, dtype, "draft", draft, "pad", pad, shift)
    with fi.DraftCheck(*(handle or (B, N)), V, DT[dtype][1], scale, draft_scale, stream()) as op:
        args = dict(draft=dev(dr) if draft and N else None, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
        a = (dev(target), tokens.cuda(), u.cuda(), r.cuda())
        op.run(*a, out, kept, lp, **args)
        torch.cuda.synchronize()
        out2, kept2 = torch.empty_like(out), torch.empty_like(kept)
        op.run(*a, out2, kept2, **args)
        torch.cuda.synchronize()
    assert torch.equal(kept.cpu(), want[1]), (kept.cpu(), want[1])
    assert torch.equal(out.cpu(), want[0])
    assert torch.equal(out, out2) and torch.equal(kept, kept2)
    g, w = lp.cpu().double(), want[2]
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    ok = torch.isnan(w) | ((g - w).abs() <= 2.0 ** -24 * w.abs() + 1e-11) | (g == w)
    assert bool(ok.all())
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 255, 256, 2047, 2048, 2049, 5000, 50001])
def test_vocabularies(V, draft, dtype):
    check(inputs(V, 6, 3, V, dtype), dtype, draft=draft)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N", [(1, 0), (1, 1), (3, 0), (200, 1), (2, 63), (40, 5), (1500, 2)])
def test_rows_and_drafts(B, N, dtype):
    check(inputs(B + N, B, N, 300, dtype), dtype)


def test_a_large_vocabulary():
    for dtype in DT:
        check(inputs(5, 3, 2, 200003, dtype), dtype)
        check(inputs(6, 1, 1, 1 << 19, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [True, False])
def test_ragged_rows(draft, dtype):
    lens = [5, 0, 1, 4, -2, 100, 3, 2]
    check(inputs(7, 8, 5, 3000, dtype, near=0.05), dtype, draft=draft, lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(61, 0), (3, 1), (64, 8)])
def test_layouts(pad, shift, dtype):
    check(inputs(8, 5, 4, 4100, dtype), dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_tokens(dtype):
    check(inputs(9, 8, 4, 3000, dtype, masked=0.9), dtype)
    x = inputs(10, 8, 4, 3000, dtype, masked=0.999)
    check(x, dtype)
    check(x, dtype, draft=False)
    x[0][:, :, :] = -math.inf
    x[0][:, :, 2500] = -5000.0 if dtype == "f32" else -4992.0    # one token, far down, in a part of its own
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_no_distribution(dtype):
    t, d, x, u, r = inputs(11, 9, 3, 2500, dtype, near=0.0)
    u = u * 0.5                                   # equal probabilities: all kept but for what follows
    t[0, 0, 100] = math.nan
    t[1, 1, 2499] = math.inf
    t[2, 2] = -math.inf
    t[3, 3, 0] = math.nan
    d[4, 1, 7] = math.nan
    d[5, 0] = -math.inf
    x[6, 2] = -1
    x[7, 0] = 2500
    x[8, 1] = 1 << 40
    want = check((t, d, x, u, r), dtype)
    assert want[1].tolist() == [0, 1, 2, 3, 1, 0, 2, 0, 1]
    assert want[0][torch.arange(4), want[1][:4].long()].tolist() == [-1] * 4
    check((t, d, x, u, r), dtype, draft=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_distributions(dtype):
    """The draft model is the target: drafts are kept whatever u below one is; a draft that both rule out
    is not, nothing is left of p - q, and the token comes from p."""
    t, d, x, u, r = inputs(12, 6, 3, 6000, dtype, near=0.0)
    t[0, 1, 55] = d[0, 1, 55] = -math.inf
    x[0, 1] = 55
    u[:] = 1.0 - 2.0 ** -24
    want = check((t, d, x, u, r), dtype)
    assert want[1].tolist() == [1, 3, 3, 3, 3, 3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r", [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0])
def test_ends_of_the_random_numbers(r, dtype):
    """r at and beyond the ends takes the first and the last token that there is."""
    t, d, x, u, _ = inputs(13, 4, 2, 4099, dtype, masked=0.5)
    t[..., :64] = -math.inf
    t[..., -64:] = -math.inf
    t[..., 700] = 1.0
    u[0] = 1.0
    u[1] = 0.0
    check((t, d, x, u, torch.full((4,), r)), dtype)
    check((t, d, x, u, torch.full((4,), r)), dtype, draft=False)


def test_borders_between_tokens():
    """r on the border of two tokens, from below and on it: 8 equal tokens, borders at eighths."""
    V = 8
    t = torch.zeros(16, 1, V)
    r = torch.tensor([x for i in range(8) for x in (i / 8, math.nextafter((i + 1) / 8, 0.0) - 2.0 ** -25)])
    out = torch.empty(16, 1, dtype=torch.int64, device="cuda")
    kept = torch.empty(16, dtype=torch.int32, device="cuda")
    z = torch.zeros(16, 0, device="cuda")
    with fi.DraftCheck(16, 0, V, fi.FI_F32, stream=stream()) as op:
        op.run(t.cuda(), z.long(), z, r.cuda(), out, kept)
        torch.cuda.synchronize()
    assert out[:, 0].tolist() == [i // 2 for i in range(16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,draft_scale", [(0.5, 2.0), (1e-6, 1e-3), (1e6, 1.0), (3e38, 3e38)])
def test_scales(scale, draft_scale, dtype):
    check(inputs(14, 4, 3, 3000, dtype), dtype, scale=scale, draft_scale=draft_scale)


def test_large_logits():
    t, d, x, u, r = inputs(15, 4, 3, 3000, "f32")
    check((t * 1e30, d * 1e30, x, u, r), "f32")
    check((t + 1e4, d + 1e4, x, u, r), "f32")
    t[..., 5] = -3.4e38
    check((t, d, x, u, r), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_on_a_larger_handle(dtype):
    for B, N in ((1, 1), (1, 7), (9, 3), (30, 0)):
        check(inputs(16, B, N, 30000, dtype), dtype, handle=(64, 8))
        check(inputs(16, B, N, 30000, dtype), dtype, draft=False, handle=(64, 8))


def test_the_target_s_distribution_comes_out():
    """What comes out first is distributed as the target's, whatever the drafts: 200000 rows of 6
    tokens; a share p is off by 5 sqrt(p / 200000) at most (5 standard deviations)."""
    B, V, g = 200000, 6, gen(17)
    p, q = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(torch.randn(V, generator=g), 0)
    x = torch.multinomial(q, B, replacement=True, generator=g)[:, None].cuda()
    out = torch.empty(B, 2, dtype=torch.int64, device="cuda")
    kept = torch.empty(B, dtype=torch.int32, device="cuda")
    t = p.log().cuda().expand(B, 2, V)
    d = q.log().cuda().expand(B, 1, V)
    with fi.DraftCheck(B, 1, V, fi.FI_F32, stream=stream()) as op:
        op.run(t, x, torch.rand(B, 1, generator=g).cuda(), torch.rand(B, generator=g).cuda(), out, kept, draft=d)
        torch.cuda.synchronize()
    share = torch.bincount(out[:, 0].cpu(), minlength=V).double() / B
    assert bool(((share - p).abs() <= 5 * torch.sqrt(p.double() / B)).all())
    assert abs(float(kept.float().mean()) - float(torch.minimum(p, q).sum())) <= 5 / math.sqrt(B)


def test_replays_of_a_graph():
    t, d, x, u, r = (y.cuda() for y in inputs(18, 8, 3, 9000, "bf16"))
    out, kept, lp = (torch.empty(8, 4, dtype=torch.int64, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda"),
                     torch.empty(8, 4, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with fi.DraftCheck(8, 3, 9000, fi.FI_BF16, stream=s) as op, torch.cuda.stream(s):
        op.run(t, x, u, r, out, kept, lp, draft=d)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            op.run(t, x, u, r, out, kept, lp, draft=d)
        for i in range(3):
            u.uniform_()
            r.uniform_()
            g.replay()
            s.synchronize()
            got = [y.clone() for y in (out, kept, lp)]
            op.run(t, x, u, r, out, kept, lp, draft=d)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (out, kept, lp)))
    torch.cuda.synchronize()


def test_refusals():
    z = torch.zeros(2, 3, 50, device="cuda")
    x, u, r = torch.zeros(2, 2, dtype=torch.int64, device="cuda"), torch.zeros(2, 2, device="cuda"), torch.zeros(2, device="cuda")
    out, kept = torch.empty(2, 3, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    with fi.DraftCheck(2, 2, 50, fi.FI_F32, stream=stream()) as op:
        def refused(*a, **kw):
            with pytest.raises(fi.FiError) as e:
                op.run(*a, **kw)
            assert e.value.status == fi.FI_ERR_INVALID
        refused(z[..., :49], x, u, r, out, kept)
        refused(z.bfloat16(), x, u, r, out, kept)
        refused(z, x[:, :1], u, r, out, kept)
        refused(z, x.int(), u, r, out, kept)
        refused(z, x, u, r.double(), out, kept)
        refused(z, x, u, r, out[:, :2], kept)
        refused(z, x, u, r, out, kept, draft=z)
        refused(z.cpu(), x, u, r, out, kept)
        refused(torch.zeros(2, 50, 3, device="cuda").transpose(1, 2), x, u, r, out, kept)
        refused(torch.zeros(3, 3, 50, device="cuda"), x, u, r, out, kept)
        refused(torch.zeros(2, 4, 50, device="cuda"), *(torch.zeros(2, 3, dtype=y, device="cuda") for y in (torch.int64, torch.float32)), r,
                torch.empty(2, 4, dtype=torch.int64, device="cuda"), kept)
        op.run(z, x, u, r, out, kept, draft=z[:, :2])
        op.run(z[:0], x[:0], u[:0], r[:0], out[:0], kept[:0])
        torch.cuda.synchronize()
