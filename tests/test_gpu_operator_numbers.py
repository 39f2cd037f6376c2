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
