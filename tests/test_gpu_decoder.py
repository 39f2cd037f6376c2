"""The decoder of examples/decoder.py, all operators together: scores of a
prompt and of the tokens after it against a plain 64-bit run of the same
weights, and the prompt's against the same tokens one at a time.

Tolerances, relative to the logits' spread (their standard
deviation): a value is rounded about 8 times a layer and 4 outside (stream, products,
attention's operands and result), each by at most u = 2^-9 (bf16) of its
size, independently, and the stream's later parts carry earlier errors on with
a gain near one: sqrt(8 * 2 + 4) u = 0.009 rms, and a maximum over some
thousand scores of five times that, 0.044, doubled for what the products'
gain adds: 0.09.  fp32: 2^-24 sqrt(K) = 2e-6 for each product's sum, by the same
reckoning 5 * sqrt(20) * 2e-6 * 2 = 9e-5, and the convolution's 1e-5.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from examples.decoder import Decoder, make_weights  # noqa: E402
from op_reference import lattn  # noqa: E402

V, D, LAYERS, H, HKV, DH, HIDDEN, B, P, N = 1000, 128, 2, 4, 2, 32, 256, 3, 150, 20
TOL = {torch.bfloat16: 0.09, torch.float32: 1e-4}


def plain(p, tokens):
    """Log probabilities [B, T, V] of every next token, in 64 bits."""
    w = {n: t.double() for n, t in p.items()}
    x = w["emb"][tokens]
    T = tokens.shape[1]
    c = torch.zeros_like(x)
    for s in range(T):
        c[:, s:] += w["filter"][s] * x[:, :T - s]
    x = x + c @ w["out"].t()
    for i in range(LAYERS):
        qkv = torch.tanh(x @ w[f"{i}.qkv"].t()).view(tokens.shape[0], T, H + 2 * HKV, DH)
        o, _ = lattn(qkv[:, :, :H], qkv[:, :, H:H + HKV], qkv[:, :, H + HKV:], p[f"{i}.decay"], 1 / math.sqrt(DH),
                     torch.zeros(tokens.shape[0], HKV, DH, DH))
        x = x + o.reshape(*x.shape[:2], -1) @ w[f"{i}.o"].t()
        u = x @ w[f"{i}.up"].t() + w[f"{i}.bias"]
        x = x + (0.5 * u * (1 + torch.erf(u / math.sqrt(2)))) @ w[f"{i}.down"].t()
    return torch.log_softmax(x @ w["head"].t(), -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens(dtype):
    weights = make_weights(V, D, LAYERS, H, HKV, DH, HIDDEN, P + N, dtype, seed=1)
    tokens = torch.randint(V, (B, P + N), generator=torch.Generator().manual_seed(2))
    ref = plain(weights, tokens)
    tol = TOL[dtype] * float(ref.std())
    given = tokens.cuda()

    whole = Decoder(weights, B, P + N, P, H, HKV, DH)
    logprob, entropy, top, ids = (t.view(B, P, *t.shape[1:]).cpu().double() for t in whole.prompt(given[:, :P]))
    want = torch.gather(ref[:, :P - 1], 2, tokens[:, 1:P, None])[..., 0]
    assert float((logprob[:, :-1] - want).abs().max()) <= tol
    assert not bool(logprob[:, -1].any())                       # no target there
    ent = -(ref.exp() * ref).sum(-1)
    assert float((entropy - ent[:, :P]).abs().max()) <= tol
    chosen = torch.gather(ref[:, :P], 2, ids.long())            # ties within the error may change places
    assert float((top - chosen).abs().max()) <= tol

    single = Decoder(weights, B, P + N, 1, H, HKV, DH)
    for t in range(P + N):
        one = single.prompt(given[:, :1]) if t == 0 else single.step(given[:, t])
        got = [one]
        if t >= P:
            got.append(whole.step(given[:, t]))
        elif t == P - 1:
            got.append((None, *(x.cuda() for x in (entropy[:, -1], top[:, -1], ids[:, -1].long()))))
        for _, e, tp, i in got:
            assert float((e.cpu().double() - ent[:, t]).abs().max()) <= tol
            assert float((tp.cpu().double() - torch.gather(ref[:, t], 1, i.cpu())).abs().max()) <= tol
    whole.close()
    single.close()
