"""Plain 64-bit forms (CPU, torch) of the gated delta rule, of normed and turned
heads and of the check of drafted tokens.  Test infrastructure."""
from __future__ import annotations

import math

import torch


def delta(q, k, v, log_decay, beta, scale, state, lens=None, slots=None, fresh=False, hold=False):
    """(o, state) in fp64, position by position; inputs on the CPU, state [slots, Hv, dk, dv]."""
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    head = torch.arange(Hv) // (Hv // Hk)
    q, k, v = q.double()[:, :, head], k.double()[:, :, head], v.double()
    a, beta = torch.exp(log_decay.double()), beta.double()
    o = torch.zeros(B, L, Hv, dv, dtype=torch.float64)
    state = state.double().clone()
    for b in range(B):
        at = b if slots is None else int(slots[b])
        if at < 0 or at >= state.shape[0]:
            continue
        n = L if lens is None else max(0, min(L, int(lens[b])))
        S = torch.zeros(Hv, dk, dv, dtype=torch.float64) if fresh else state[at].clone()
        for t in range(n):
            S = torch.where(a[b, t][:, None, None] > 0, a[b, t][:, None, None] * S, 0.0)
            u = beta[b, t][:, None] * (v[b, t] - (k[b, t][..., None] * S).sum(1))
            S = S + k[b, t][..., None] * u[:, None]
            o[b, t] = scale * (q[b, t][..., None] * S).sum(1)
        if not hold:
            state[at] = S
    return o, state


def rotary(x, w, where, inv_freq, norm, eps, adjacent):
    """Heads x [B, L, H, d] normed, weighted and turned at the positions where [B, L], in fp64."""
    x = x.double()
    if norm:
        s = x.square().sum(-1, keepdim=True)
        x = x / torch.sqrt((s / x.shape[-1] if norm == 1 else s) + eps)
    if w is not None:
        x = x * w.double()
    y = x.clone()
    for i in range(len(inv_freq)):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + len(inv_freq))
        angle = (where.double() * float(inv_freq[i]))[..., None]
        c, s = torch.cos(angle), torch.sin(angle)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def verify(target, draft, tokens, lens, u, r, scale=1.0, draft_scale=1.0):
    """(out, kept, logprob) by the header's rules, in fp64; draft may be None."""
    B, N = tokens.shape
    V = target.shape[2]
    out = torch.full((B, N + 1), -1, dtype=torch.int64)
    kept = torch.zeros(B, dtype=torch.int32)
    lp = torch.zeros(B, N + 1, dtype=torch.float64)

    def dist(z, c):
        z = z.double() * c
        if bool(torch.isnan(z).any()) or bool((z == math.inf).any()) or not bool((z > -math.inf).any()):
            return None, None
        e = torch.exp(z - z.max())
        return e / e.sum(), (z - z.max()) - torch.log(e.sum())
    for b in range(B):
        n = N if lens is None else max(0, min(N, int(lens[b])))
        i = 0
        while i < n:
            x = int(tokens[b, i])
            p, logp = dist(target[b, i], scale)
            if p is None or not 0 <= x < V:
                break
            qx = 1.0
            if draft is not None:
                q, _ = dist(draft[b, i], draft_scale)
                if q is None:
                    break
                qx = float(q[x])
            if not float(u[b, i]) * qx < float(p[x]):
                break
            out[b, i], lp[b, i] = x, logp[x]
            i += 1
        kept[b] = i
        p, logp = dist(target[b, i], scale)
        if p is None:
            lp[b, i] = math.nan
            continue
        w = p
        if i < n:
            if draft is None:
                w = p.clone()
                if 0 <= int(tokens[b, i]) < V:
                    w[int(tokens[b, i])] = 0.0
            else:
                q, _ = dist(draft[b, i], draft_scale)
                w = p if q is None else (p - q).clamp(min=0.0)
            if not float(w.sum()) > 0.0:
                w = p
        ids = torch.nonzero(w > 0)[:, 0]
        sums = w[ids].cumsum(0)
        hit = torch.nonzero(sums > float(r[b]) * sums[-1])
        out[b, i] = ids[int(hit[0]) if len(hit) else -1]
        lp[b, i] = logp[out[b, i]]
    return out, kept, lp
