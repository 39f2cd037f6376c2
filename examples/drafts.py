"""A decoder that answers with drafted tokens, on the library's operators: layers of
the gated delta rule with normed and turned heads, blocks, a head, and a check of
several drafted tokens at a time.

    python examples/drafts.py [--rows 4] [--prompt 256] [--rounds 32] [--drafts 4]

Every position x of the residual stream goes through, in each layer,

    q, k, v = tanh(qkv . x)                       Dense
    q, k = turned(normed(q)), turned(normed(k))   Rotary (length one, as the delta rule wants its keys)
    a, beta = gates(gate . x)                     Dense
    x += o . delta(q, k, v, a, beta)              DeltaRule, Dense
    x += down . gelu(up . x)                      Dense, Dense

A round of answering: a small model drafts N tokens, the large one runs over all of them
with its states held, DraftCheck keeps some and draws one more, and the states move over
what was kept, whose keys and values are still there.  How many were kept stays on
the device: nothing waits for it.  Weights are random.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_online_amd as fi  # noqa: E402


def make_weights(V, D, layers, Hk, Hv, dh, hidden, dtype, seed=0):
    """Random weights on the CPU, {name: tensor}; products scaled to keep the stream's size."""
    g = torch.Generator().manual_seed(seed)

    def w(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g) * (gain / math.sqrt(shape[-1]))).to(dtype)
    p = {"emb": torch.randn(V, D, generator=g).to(dtype), "head": w(V, D)}
    for i in range(layers):
        p |= {f"{i}.qkv": w((2 * Hk + Hv) * dh, D), f"{i}.gate": w(2 * Hv, D), f"{i}.o": w(D, Hv * dh, gain=0.5),
              f"{i}.up": w(hidden, D), f"{i}.down": w(D, hidden, gain=0.5)}
    return p


def gates(x):
    """(log_decay, beta) of the gates' product x [..., 2 Hv]: decays of e^-0.0002 to e^-0.7 a position, beta in (0, 1)."""
    a, b = x.chunk(2, -1)
    return -torch.nn.functional.softplus(a - 4.0), torch.sigmoid(b)


class DeltaDecoder:
    """B rows, calls of at most L positions; states stay with the rows."""

    def __init__(self, weights, B, L, Hk, Hv, dh, stream=None):
        s = stream or torch.cuda.current_stream()
        p = self.p = {n: t.cuda() for n, t in weights.items()}
        self.B, self.L, self.Hk, self.Hv, self.dh = B, L, Hk, Hv, dh
        self.V, self.D = p["emb"].shape
        self.layers = sum(n.endswith(".qkv") for n in p)
        dtype = p["emb"].dtype
        io = fi.FI_BF16 if dtype == torch.bfloat16 else fi.FI_F32
        rows = B * L

        def dense(name):
            N, K = p[name].shape
            act = {"qkv": fi.FI_ACT_TANH, "up": fi.FI_ACT_GELU}.get(name.split(".")[-1], fi.FI_ACT_IDENTITY)
            return fi.Dense(rows, N, K, io, fi.FI_F32 if name == "head" or name.endswith(".gate") else io, act, stream=s)
        self.dense = {n: dense(n) for n in p if n != "emb"}
        freq = (1e4 ** (-torch.arange(dh // 4) * 4.0 / dh)).float().cuda()      # half of a head is turned
        self.turn = fi.Rotary(B, L, Hk, Hk, dh, freq, fi.FI_NORM_L2, 1e-6, io_dtype=io, stream=s)
        self.mix = fi.DeltaRule(B, L, Hk, Hv, dh, dh, 1.0, io, stream=s)         # one workspace for all layers: the states are ours
        self.state = [torch.zeros(B, Hv, dh, dh, device="cuda") for _ in range(self.layers)]
        self.at = torch.zeros(B, dtype=torch.int32, device="cuda")               # where the rows' next positions stand
        empty = lambda *shape, t=dtype: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
        self.x, self.att, self.logits = empty(rows, self.D), empty(rows, Hv * dh), empty(rows, self.V, t=torch.float32)
        self.hid = empty(rows, p["0.up"].shape[0])
        # a layer's own, as the states may move over them later
        self.qkv = [empty(rows, (2 * Hk + Hv) * dh) for _ in range(self.layers)]
        self.gate = [(empty(rows, 2 * Hv, t=torch.float32), None, None) for _ in range(self.layers)]

    def _heads(self, i, T):
        h = self.qkv[i][:self.B * T].view(self.B, T, 2 * self.Hk + self.Hv, self.dh)
        return h[:, :, :self.Hk], h[:, :, self.Hk:2 * self.Hk], h[:, :, 2 * self.Hk:]

    def run(self, tokens, lens=None, fresh=False, hold=False):
        """Logits [B, T, V] of the positions tokens [B, T].  The states move over them (over the first lens of each row), or, held, stay."""
        p, B, T = self.p, self.B, tokens.shape[1]
        n = B * T
        x, att, hid, logits = (t[:n] for t in (self.x, self.att, self.hid, self.logits))
        if fresh:
            self.at.zero_()
        torch.index_select(p["emb"], 0, tokens.reshape(-1), out=x)
        for i in range(self.layers):
            raw = self.gate[i][0][:n]
            self.dense[f"{i}.qkv"].run(x, p[f"{i}.qkv"], self.qkv[i][:n])
            self.dense[f"{i}.gate"].run(x, p[f"{i}.gate"], raw)
            q, k, v = self._heads(i, T)
            self.turn.run(q, k, q, k, first=self.at)
            a, b = gates(raw.view(B, T, -1))
            self.gate[i] = (self.gate[i][0], a, b)
            self.mix.prompt(q, k, v, a, b, att.view(B, T, self.Hv, self.dh), self.state[i], lens=lens, fresh=fresh, hold=hold)
            self.dense[f"{i}.o"].run(att, p[f"{i}.o"], x, res=x)
            self.dense[f"{i}.up"].run(x, p[f"{i}.up"], hid)
            self.dense[f"{i}.down"].run(hid, p[f"{i}.down"], x, res=x)
        self.dense["head"].run(x, p["head"], logits)
        if not hold:
            self.at += T if lens is None else lens
        return logits.view(B, T, self.V)

    def move(self, T, lens):
        """After a held run over T positions: the states move over the first lens [B] of them."""
        att = self.att[:self.B * T].view(self.B, T, self.Hv, self.dh)
        for i in range(self.layers):
            self.mix.prompt(*self._heads(i, T), *self.gate[i][1:], att, self.state[i], lens=lens)
        self.at += lens

    def close(self):
        for h in (self.turn, self.mix, *self.dense.values()):
            h.close()


class Answer:
    """Rounds of N drafts by `small`, checked by `large`; both have run over the prompt but its last token."""

    def __init__(self, large, small, N, stream=None):
        self.large, self.small, self.N = large, small, N
        B, V = large.B, large.V
        self.check = fi.DraftCheck(B, N, V, fi.FI_F32, stream=stream or torch.cuda.current_stream())
        self.tokens = torch.empty(B, N + 1, dtype=torch.int64, device="cuda")     # the last known token, and the drafts
        self.drafts = torch.empty(B, N, V, device="cuda")
        self.out = torch.empty(B, N + 1, dtype=torch.int64, device="cuda")
        self.kept = torch.empty(B, dtype=torch.int32, device="cuda")
        self.logprob = torch.empty(B, N + 1, device="cuda")

    def round(self, last, noise, u, r):
        """One round behind the tokens `last` [B]: noise [B, N, V] (uniform) draws the drafts, u [B, N] and r [B] check
        them.  (out, kept, logprob): kept + 1 new tokens of each row in out, then -1."""
        small, N = self.small, self.N
        self.tokens[:, 0] = last
        states = [s.clone() for s in small.state]                                # to come back to
        at = small.at.clone()
        for i in range(N):
            z = small.run(self.tokens[:, i:i + 1].contiguous())[:, 0]
            self.drafts[:, i] = z
            self.tokens[:, i + 1] = (z - torch.log(-torch.log(noise[:, i].clamp(1e-20, 1.0 - 6e-8)))).argmax(-1)
        for s, old in zip(small.state, states):
            s.copy_(old)
        small.at.copy_(at)
        z = self.large.run(self.tokens, hold=True)
        self.check.run(z, self.tokens[:, 1:].contiguous(), u, r, self.out, self.kept, self.logprob, draft=self.drafts)
        moved = self.kept + 1
        self.large.move(N + 1, moved)
        small.run(self.tokens, lens=moved)
        return self.out, self.kept, self.logprob

    def last(self):
        """The newest token of every row."""
        return self.out.gather(1, self.kept.long()[:, None])[:, 0].clamp(min=0)   # (-1, of rows without any, is no place in the embeddings)

    def close(self):
        self.check.close()


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=256)
    ap.add_argument("--rounds", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    V, D, Hk, Hv, dh, hidden, L = 32768, 1024, 8, 16, 64, 4096, max(a.prompt, a.drafts + 1)
    weights = make_weights(V, D, 4, Hk, Hv, dh, hidden, torch.bfloat16)
    large = DeltaDecoder(weights, a.rows, L, Hk, Hv, dh)
    small = DeltaDecoder({n: t for n, t in weights.items() if n[0] in "eh0"}, a.rows, L, Hk, Hv, dh)   # its first layer
    prompt = torch.randint(V, (a.rows, a.prompt), device="cuda")
    ans = Answer(large, small, a.drafts)
    for _ in range(2):   # the second time is the warm one
        for m in (large, small):
            m.run(prompt[:, :-1].contiguous(), fresh=True)
        last, new = prompt[:, -1], torch.zeros(a.rows, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.rounds):
            rand = torch.rand(a.rows, a.drafts * V + a.drafts + 1, device="cuda")
            noise, u, r = rand.split([a.drafts * V, a.drafts, 1], 1)
            ans.round(last, noise.view(a.rows, a.drafts, V), u.contiguous(), r[:, 0].contiguous())
            last, new = ans.last(), new + ans.kept + 1
        torch.cuda.synchronize()
        t1 = time.perf_counter()
    print(f"{a.rounds} rounds of {a.drafts} drafts, {a.rows} rows: {(t1 - t0) / a.rounds * 1e3:.2f} ms a round, "
          f"{float(new.mean()) / a.rounds:.2f} tokens a row and round; first row's last: {ans.out[0].tolist()}")
    for h in (ans, large, small):
        h.close()


if __name__ == "__main__":
    main()
