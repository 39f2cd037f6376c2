"""A small decoder on the library's operators: a long convolution, layers of
linear attention with blocks, a head, and the scores of its tokens.

    python examples/decoder.py [--tokens 64] [--prompt 512] [--rows 4]

Every position x of the residual stream goes through

    x += out . conv(x)                            Mixer (fi_step), Dense
    x += o . attention(tanh(qkv . x))             Dense, LinearAttention, Dense
    x += down . gelu(up . x + bias)               Dense, Dense      (each layer)
    scores(head . x)                              Dense, TokenScores

A prompt runs the products and the attention over all of its positions at
once; a generated token runs the recurrent form over the same states.  torch
holds the memory and gathers the embeddings; nothing waits for the device
between tokens (the next one is chosen there).  Weights are random.
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


def make_weights(V, D, layers, H, Hkv, dh, hidden, L, dtype, seed=0):
    """Random weights on the CPU, {name: tensor}; products scaled to keep the stream's size."""
    g = torch.Generator().manual_seed(seed)

    def w(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g) * (gain / math.sqrt(shape[-1]))).to(dtype)
    p = {"emb": torch.randn(V, D, generator=g).to(dtype), "head": w(V, D), "out": w(D, D, gain=0.5),
         "filter": (torch.randn(L, D, generator=g) * (0.5 / (1.0 + torch.arange(L))[:, None])).to(dtype)}
    for i in range(layers):
        p |= {f"{i}.qkv": w((H + 2 * Hkv) * dh, D), f"{i}.o": w(D, H * dh, gain=0.5), f"{i}.up": w(hidden, D),
              f"{i}.bias": (0.1 * torch.randn(hidden, generator=g)).to(dtype), f"{i}.down": w(D, hidden, gain=0.5),
              f"{i}.decay": -torch.exp2(-1.0 - 6.0 * torch.rand(Hkv, generator=g))}
    return p


class Decoder:
    """B rows over at most L positions; prompt() once, then step()."""

    def __init__(self, weights, B, L, prompt, H, Hkv, dh, k=4):
        s = torch.cuda.current_stream()
        p = self.p = {n: t.cuda() for n, t in weights.items()}
        self.B, self.H, self.Hkv, self.dh, self.k = B, H, Hkv, dh, k
        self.V, self.D = p["emb"].shape
        self.layers = sum(n.endswith(".qkv") for n in p)
        dtype = p["emb"].dtype
        io = fi.FI_BF16 if dtype == torch.bfloat16 else fi.FI_F32
        rows = B * max(prompt, 1)
        self.conv = fi.Mixer(B, self.D, L, p["filter"], io_dtype=io, stream=s)

        def dense(name, out=io, act=fi.FI_ACT_IDENTITY):
            N, K = p[name].shape
            return fi.Dense(rows, N, K, io, out, act, stream=s)
        # tanh bounds q, k and v: their products would grow with the cube of the stream
        acts = {"qkv": fi.FI_ACT_TANH, "up": fi.FI_ACT_GELU}
        self.dense = {n: dense(n, act=acts.get(n.split(".")[-1], fi.FI_ACT_IDENTITY))
                      for n in p if n == "out" or n.split(".")[-1] in ("qkv", "o", "up", "down")}
        self.dense["head"] = dense("head", out=fi.FI_F32)
        scale = 1.0 / math.sqrt(dh)
        self.mix = [fi.LinearAttention(B, max(prompt, 1), H, Hkv, dh, dh, p[f"{i}.decay"], scale, io, stream=s)
                    for i in range(self.layers)]
        self.state = [torch.zeros(B, Hkv, dh, dh, device="cuda") for _ in range(self.layers)]
        self.scorer = fi.TokenScores(rows, self.V, k, fi.FI_F32, stream=s)
        empty = lambda *shape, t=dtype: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
        hidden = p["0.up"].shape[0] if self.layers else 1
        self.x, self.c = empty(rows, self.D), empty(rows, self.D)
        self.xt, self.ct = empty(B, self.D), empty(B, self.D, t=torch.float32)
        self.qkv, self.att = empty(rows, (H + 2 * Hkv) * dh), empty(rows, H * dh)
        self.hid, self.logits = empty(rows, hidden), empty(rows, self.V, t=torch.float32)

    def _run(self, tokens, targets, fresh):
        """tokens [B, T] -> (logprob of targets or None, entropy, top, top_id), B * T rows."""
        p, B, T = self.p, self.B, tokens.shape[1]
        n, H, Hkv, dh = B * T, self.H, self.Hkv, self.dh
        x, c, qkv, att, hid, logits = (t[:n] for t in (self.x, self.c, self.qkv, self.att, self.hid, self.logits))
        torch.index_select(p["emb"], 0, tokens.reshape(-1), out=x)
        for t in range(T):
            self.xt.copy_(x.view(B, T, -1)[:, t])
            self.conv.step(self.xt, self.ct)
            c.view(B, T, -1)[:, t].copy_(self.ct)
        self.dense["out"].run(c, p["out"], x, res=x)
        heads = qkv.view(B, T, H + 2 * Hkv, dh)
        q, kk, v, o = heads[:, :, :H], heads[:, :, H:H + Hkv], heads[:, :, H + Hkv:], att.view(B, T, H, dh)
        for i in range(self.layers):
            self.dense[f"{i}.qkv"].run(x, p[f"{i}.qkv"], qkv)
            if fresh:
                self.mix[i].prompt(q, kk, v, o, self.state[i], fresh=True)
            else:
                self.mix[i].step(q, kk, v, o, self.state[i])
            self.dense[f"{i}.o"].run(att, p[f"{i}.o"], x, res=x)
            self.dense[f"{i}.up"].run(x, p[f"{i}.up"], hid, bias=p[f"{i}.bias"])
            self.dense[f"{i}.down"].run(hid, p[f"{i}.down"], x, res=x)
        self.dense["head"].run(x, p["head"], logits)
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        entropy, top, ids = f32(n), f32(n, self.k), torch.empty(n, self.k, dtype=torch.int64, device="cuda")
        logprob = None if targets is None else f32(n)
        self.scorer.run(logits, None if targets is None else targets.reshape(-1), logprob, entropy, top, ids)
        return logprob, entropy, top, ids

    def prompt(self, tokens):
        """Scores of tokens [B, T] (int64); the last position has no target."""
        targets = torch.full_like(tokens, -1)
        targets[:, :-1] = tokens[:, 1:]
        self.conv.reset()
        return self._run(tokens, targets, True)

    def step(self, tokens):
        """Scores after one more token of every row, tokens [B]."""
        return self._run(tokens.view(self.B, 1), None, False)

    @staticmethod
    def best(ids):
        """The most probable token of every row of alternatives [rows, k]; 0 where a row has none
        (its -1 is no place in the embeddings)."""
        return ids[:, 0].clamp(min=0)

    def close(self):
        for h in (self.conv, self.scorer, *self.mix, *self.dense.values()):
            h.close()


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    V, D, layers, H, Hkv, dh, hidden = 32768, 1024, 4, 16, 8, 64, 4096
    L = a.prompt + a.tokens
    d = Decoder(make_weights(V, D, layers, H, Hkv, dh, hidden, L, torch.bfloat16), a.rows, L, a.prompt, H, Hkv, dh)
    tokens = torch.randint(V, (a.rows, a.prompt), device="cuda")
    for _ in range(2):   # the second time is the warm one
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        logprob, entropy, _, ids = d.prompt(tokens)
        torch.cuda.synchronize()
        t1 = time.perf_counter()
        last, out = d.best(ids.view(a.rows, a.prompt, -1)[:, -1]), []
        for _ in range(a.tokens):
            out.append(last)
            last = d.best(d.step(last)[3])
        torch.cuda.synchronize()
        t2 = time.perf_counter()
    print(f"prompt of {a.rows} x {a.prompt}: {(t1 - t0) * 1e3:.2f} ms, mean log probability {float(logprob.mean()):.3f}, "
          f"mean entropy {float(entropy.mean()):.3f}")
    print(f"{a.tokens} tokens a row: {(t2 - t1) * 1e3:.2f} ms, {(t2 - t1) / a.tokens * 1e6:.0f} us each; first row: "
          f"{torch.stack(out, 1)[0, :8].tolist()}")
    d.close()


if __name__ == "__main__":
    main()
