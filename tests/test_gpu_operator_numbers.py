"""Where the operators' numbers can be off without being far off: single rows
and heads, the tails of an activation, sums of very many terms, scales at the
ends of fp32's range.  Each bound stands with its derivation."""
import math

import pytest

import op_reference as ref
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


# ------------------------------------------------------------ linear attention
@pytest.mark.parametrize("H,Hkv,dk,dv,L,fresh", [
    (4, 2, 64, 64, 77, True), (4, 4, 64, 40, 300, False), (4, 2, 128, 128, 200, False), (2, 1, 100, 70, 2100, False),
    (3, 3, 33, 7, 150, True), (2, 1, 256, 192, 130, False), (16, 2, 48, 80, 64, True)])
def test_prompt_bf16_is_rounded_once(H, Hkv, dk, dv, L, fresh):
    """A bf16 output is the formula's value rounded to bf16, of every row and head.

    The products' operands are bf16, so an fp32 factor enters as two bf16
    parts: off by 2^-15 of it at most, 2^-17 in the mean square; with the fp32
    sums, whose terms may be 2^5 times their sum, the value before its rounding is
    off by d <= 2^-12 of o.  That turns a share of 2 d / 2^-8 of the
    roundings over, each by a step of at most 2^-7 of o: relative L2 distance from the
    rounded value <= sqrt(d 2^-7) < 2^-9.5 = 1.4e-3.  (Factors of one bf16
    part, 2^-9 in the mean square, would be off by more than 2e-3.)"""
    B = 2
    g = gen(H * dk + L)
    q = torch.randn(B, L, H, dk, generator=g).bfloat16()
    k = torch.randn(B, L, Hkv, dk, generator=g).bfloat16()
    v = torch.randn(B, L, Hkv, dv, generator=g).bfloat16()
    tau = torch.exp(math.log(8.0) + torch.rand(Hkv, generator=g) * math.log(512.0))
    ld = -1.0 / tau
    state = torch.randn(B, Hkv, dk, dv, generator=g) * tau[None, :, None, None].sqrt()
    ro, rs = ref.lattn(q, k, v, ld, 0.125, state, fresh=fresh)
    o, st = torch.empty(B, L, H, dv, dtype=torch.bfloat16, device="cuda"), state.cuda()
    log("case prompt, rounded once", H, Hkv, dk, dv, L, fresh)
    with fi.LinearAttention(B, L, H, Hkv, dk, dv, ld.cuda(), 0.125, fi.FI_BF16, stream()) as op:
        op.prompt(q.cuda(), k.cuda(), v.cuda(), o, st, fresh=fresh)
        torch.cuda.synchronize()
    once = ro.bfloat16().double()
    far = [ref.rel_l2(o[b, :, h], once[b, :, h]) for b in range(B) for h in range(H)]
    log("largest distance of a row and head %.3g" % max(far))
    assert max(far) <= 2.0 ** -9.5
    assert max(ref.rel_l2(st[b, n], rs[b, n]) for b in range(B) for n in range(Hkv)) <= 5e-6


# ------------------------------------------------------------ dense product
@pytest.mark.parametrize("rows", ["one", "many"])
def test_dense_gelu_keeps_its_tails(rows):
    """GELU v Phi(v) of fp32 at v = x w, K = 1: relative in Phi(-|v|), which
    every value on the negative side is made of.

    Phi(-|v|) = e^{-v^2/2} times a polynomial: the polynomial's fit, its
    evaluation, a reciprocal and an exponential, a unit of 2^-23 each and two for the
    products, and the exponent's three roundings, 2^-24 each of v^2 / 2 log2 e:
    (6 + v^2) 2^-23; then one rounding of y.  Below 2^-125 results may be flushed."""
    v = torch.cat([torch.linspace(-14, 14, 2 * 8191 + 1), torch.tensor([0.0, -1e-6, 1e-6, 50.0, -50.0, 3e4, -3e4])])
    x, w = (torch.ones(1, 1), v[:, None]) if rows == "one" else (v[:, None], torch.ones(65, 1))
    z = x @ w.t()
    y = torch.empty_like(z, device="cuda")
    with fi.Dense(z.shape[0], z.shape[1], 1, fi.FI_F32, fi.FI_F32, fi.FI_ACT_GELU, stream()) as op:
        op.run(x.cuda(), w.cuda(), y)
        torch.cuda.synchronize()
    z = z.double()
    phi = torch.special.erfc(z.abs() / math.sqrt(2.0)) / 2   # (ndtr takes 1 + erf: 0 below -8.3)
    want = z.clamp(min=0) - z.abs() * phi
    bound = 2.0 ** -24 * want.abs() + z.abs() * phi * (6 + z * z) * 2.0 ** -23 + 2.0 ** -125 * z.abs().clamp(min=1)
    over = (y.cpu().double() - want).abs() / bound.clamp(min=1e-300)
    log("gelu, largest share of its bound %.3g at %.4g" % (over.max(), z.flatten()[over.argmax()]))
    assert float(over.max()) <= 1.0


# ------------------------------------------------------------ token scores
def run_scores(z, t, k, dtype, scale=1.0):
    R, V = z.shape
    lp, H, lse = (torch.full((R,), 9.0, device="cuda") for _ in range(3))
    top, ids = torch.empty(R, k, device="cuda"), torch.empty(R, k, dtype=torch.int64, device="cuda")
    with fi.TokenScores(R, V, k, DT[dtype][1], scale, stream()) as op:
        op.run(z, t, lp, H, top, ids, lse)
        torch.cuda.synchronize()
    return [x.cpu() for x in (lp, H, lse, top, ids)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(1100, 131072), (1030, 200000), (1, 1 << 26)])
def test_scores_of_many_equal_logits(R, V, dtype):
    """One peak at 0 over a floor of equal logits -d, a row for each of several d:
    every term of a sum rounds the same way, so sums of n terms one after the other
    would be off by up to n 2^-25 of their value (n = V / 64: 6e-5).

    Bounds as for any row: 2^t is off by |t| 2^-23, log probabilities by
    1e-6 (8 + |lp|), lse by 1e-6 (4 + |lse|), entropies by 1e-6 (4 + H)."""
    depth = [1.5, 2.5, 5.0, 5.25, 3.3125, 9.0, 11.5] if R > 1 else [2.5]
    d = torch.tensor([depth[r % len(depth)] for r in range(R)])
    z = (-d[:, None]).expand(R, V).to("cuda", DT[dtype][0]).contiguous()
    z[:, V // 3] = 0.0
    t = torch.full((R,), V - 1, dtype=torch.int64, device="cuda")
    t[::2] = V // 3
    lp, H, lse, top, ids = run_scores(z, t, 2, dtype)
    d = d.double()      # (all of them are bf16 numbers)
    rlse = torch.log1p((V - 1) * torch.exp(-d))
    rlp = torch.where(t.cpu() == V // 3, 0.0, -d) - rlse
    rH = rlse * torch.exp(-rlse) + (V - 1) * (d + rlse) * torch.exp(-d - rlse)
    for what, got, want, a in (("lse", lse, rlse, 4e-6), ("logprob", lp, rlp, 8e-6), ("entropy", H, rH, 4e-6)):
        e = (got.double() - want).abs()
        log(what, R, V, dtype, "off by %.3g" % e.max())
        assert bool((e <= a + 1e-6 * want.abs()).all()), what
    assert ids[0].tolist() == [V // 3, 0]
    assert bool(((top[:, 0].double() + rlse).abs() <= 8e-6 + 1e-6 * rlse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 40000])
@pytest.mark.parametrize("scale", [2.0e38, 3.0e38, 3.4e38])
def test_scores_of_the_largest_scales(V, scale, dtype):
    """Finite scales whose product with log2 e is not: logits that
    lie some 1e-38 apart, and ordinary ones, where all of the probability is with the
    largest.  The bounds of ordinary rows (logits below 2^-126 are whole
    multiples of 2^-149, so their differences are exact)."""
    g = gen(V)
    z = torch.randn(5, V, generator=g).to(DT[dtype][0])
    z[0] = (torch.randn(V, generator=g) * 1.5e-38).to(DT[dtype][0])
    z[1] = (torch.randn(V, generator=g) * 2.0 ** -126).to(DT[dtype][0])
    z[2] = 0.0
    z[3, V // 2] = 7.0
    t = torch.randint(0, V, (5,), generator=g)
    lp, H, lse, top, ids = run_scores(z.cuda(), t.cuda(), 6, dtype, scale)
    rlp, rH, rlse, rtop, rids = ref.scores(z, t, 6, torch.tensor(scale).item())
    assert torch.equal(ids, rids)
    for got, want, a in ((lp, rlp, 8e-6), (H, rH, 4e-6), (lse, rlse, 4e-6), (top, rtop, 8e-6)):
        f = torch.isfinite(want.float())
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~f], want.float()[~f])
        assert bool(((got.double() - want).abs()[f] <= a + 1e-6 * want.abs()[f]).all())
