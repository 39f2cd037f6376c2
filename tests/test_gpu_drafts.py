"""The operators of drafted answers together (examples/drafts.py): logits against
a plain 64-bit run of the same weights, rounds of drafts against the check's rules on the
same logits, and the states that held runs and moves leave against a prompt over the
tokens that came out.

Tolerances, relative to the spread of what is compared: fp32, each product's sum is off by
2^-24 sqrt(K) <= 2e-6 and the delta rule by 1e-5; about 8 of them in a layer, independent, with a
gain near one: sqrt(16) * 1e-5 rms over two layers, five times that for the largest of some thousand,
doubled for the products' gain: 4e-4.  bf16: 8 roundings of 2^-9 rms in a layer, sqrt(16) 2^-9 =
0.008, times ten likewise: 0.08."""
import pytest

import draft_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from examples.drafts import Answer, DeltaDecoder, gates, make_weights  # noqa: E402

V, D, LAYERS, HK, HV, DH, HIDDEN = 700, 96, 2, 2, 4, 32, 192
TOL = {torch.bfloat16: 0.08, torch.float32: 4e-4}


def plain(p, tokens):
    """Logits [B, T, V] in 64 bits, and each layer's state."""
    w = {n: t.double() for n, t in p.items()}
    x = w["emb"][tokens]
    B, T = tokens.shape
    freq = (1e4 ** (-torch.arange(DH // 4) * 4.0 / DH)).float()
    where = torch.arange(T)[None].expand(B, T)
    states = []
    for i in range(sum(n.endswith(".qkv") for n in p)):
        h = torch.tanh(x @ w[f"{i}.qkv"].t()).view(B, T, 2 * HK + HV, DH)
        q, k = (ref.rotary(y, None, where, freq, 2, 1e-6, False) for y in (h[:, :, :HK], h[:, :, HK:2 * HK]))
        a, b = gates(x @ w[f"{i}.gate"].t())
        o, s = ref.delta(q, k, h[:, :, 2 * HK:], a, b, 1.0, torch.zeros(B, HV, DH, DH))
        states.append(s)
        x = x + o.reshape(B, T, -1) @ w[f"{i}.o"].t()
        u = x @ w[f"{i}.up"].t()
        x = x + (0.5 * u * (1 + torch.erf(u / 2.0 ** 0.5))) @ w[f"{i}.down"].t()
    return x @ w["head"].t(), states


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 7, 40, 130])
def test_logits(T, dtype):
    weights = make_weights(V, D, LAYERS, HK, HV, DH, HIDDEN, dtype, seed=1)
    tokens = torch.randint(V, (3, T), generator=torch.Generator().manual_seed(T))
    want, states = plain(weights, tokens)
    m = DeltaDecoder(weights, 3, T, HK, HV, DH)
    z = m.run(tokens.cuda(), fresh=True)
    torch.cuda.synchronize()
    assert float((z.cpu().double() - want).abs().max()) <= TOL[dtype] * float(want.std())
    for s, w in zip(m.state, states):
        assert float((s.cpu().double() - w).abs().max()) <= TOL[dtype] * float(w.abs().max())
    # token by token, from the beginning
    for t in range(T):
        z = m.run(tokens[:, t:t + 1].cuda(), fresh=t == 0)
        torch.cuda.synchronize()
        assert float((z[:, 0].cpu().double() - want[:, t]).abs().max()) <= TOL[dtype] * float(want.std())
    m.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 4, 9])
def test_rounds_of_drafts(N, dtype):
    B, P, ROUNDS, g = 3, 50, 6, torch.Generator().manual_seed(N)
    weights = make_weights(V, D, LAYERS, HK, HV, DH, HIDDEN, dtype, seed=2)
    large = DeltaDecoder(weights, B, P, HK, HV, DH)
    small = DeltaDecoder({n: t for n, t in weights.items() if n[0] in "eh0"}, B, P, HK, HV, DH)
    ans = Answer(large, small, N)
    prompt = torch.randint(V, (B, P), generator=g)
    rows = [prompt[b].tolist() for b in range(B)]
    for m in (large, small):
        m.run(prompt[:, :-1].cuda().contiguous(), fresh=True)
    last, kept_in_all = prompt[:, -1].cuda(), 0
    for _ in range(ROUNDS):
        noise, u, r = torch.rand(B, N, V, generator=g), torch.rand(B, N, generator=g), torch.rand(B, generator=g)
        held = [s.clone() for s in large.state]
        out, kept, lp = ans.round(last, noise.cuda(), u.cuda(), r.cuda())
        torch.cuda.synchronize()
        z = large.logits[:B * (N + 1)].view(B, N + 1, V).cpu()
        want = ref.verify(z, ans.drafts.cpu(), ans.tokens[:, 1:].cpu(), None, u, r)
        assert torch.equal(out.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
        assert float((lp.cpu().double() - want[2]).abs().max()) <= 1e-5
        assert any(not torch.equal(a, b) for a, b in zip(held, large.state))
        for b in range(B):
            rows[b] += out[b, :int(kept[b]) + 1].tolist()
        kept_in_all += int(kept.sum())
        last = ans.last()
    assert large.at.tolist() == [len(x) - 1 for x in rows] == small.at.tolist()
    assert 0 < kept_in_all < ROUNDS * N * B
    # the states are those of the tokens that came out, but the newest
    for m in (large, small):
        for b in range(B):
            _, states = plain({n: t for n, t in weights.items() if n in m.p}, torch.tensor([rows[b][:-1]]))
            for s, w in zip(m.state, states):
                assert float((s[b].cpu().double() - w[0]).abs().max()) <= TOL[dtype] * float(w.abs().max()), b
    for h in (ans, large, small):
        h.close()
