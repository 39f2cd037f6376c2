"""Plain 64-bit forms (CPU, torch) of the operators around the mixers, and the
error bounds that the GPU tests hold the kernels to.  Test infrastructure."""
from __future__ import annotations

import math

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8      # largest relative error of a rounding to fp32 (24 bits) and bf16 (8 bits)


def rel_l2(a, b) -> float:
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    n = float(b.norm())
    d = float((a - b).norm())
    return d / n if n > 0 else d


def lattn(q, k, v, log_decay, scale, state, lens=None, slots=None, fresh=False):
    """(o, state) in fp64; inputs on the CPU, state [slots, Hkv, dk, dv]."""
    q, k, v = (x.double() for x in (q, k, v))
    B, L, H, dk = q.shape
    Hkv, dv = k.shape[2], v.shape[3]
    G = H // Hkv
    o = torch.zeros(B, L, H, dv, dtype=torch.float64)
    state = state.double().clone()
    for b in range(B):
        at = b if slots is None else int(slots[b])
        if at < 0 or at >= state.shape[0]:
            continue
        n = L if lens is None else max(0, min(L, int(lens[b])))
        for m in range(Hkv):
            ld = float(log_decay[m])
            S = torch.zeros(dk, dv, dtype=torch.float64) if fresh else state[at, m]
            i = torch.arange(n, dtype=torch.float64)
            power = lambda e: torch.where(e == 0, 1.0, torch.exp(ld * e.clamp(min=1)))  # noqa: E731
            lag = i[:, None] - i[None, :]
            w = torch.where(lag >= 0, power(lag.clamp(min=0)), 0.0)
            kk, vv = k[b, :n, m], v[b, :n, m]
            for g in range(G):
                qq = q[b, :n, m * G + g]
                o[b, :n, m * G + g] = scale * (((qq @ kk.t()) * w) @ vv + power(i + 1)[:, None] * (qq @ S))
            decay = 1.0 if n == 0 else math.exp(ld * n)
            state[at, m] = (decay * S if decay else 0.0 * S) + (kk * power(n - 1 - i)[:, None]).t() @ vv
    return o, state


def dense(x, w, bias, act, res):
    """(y, bound of the sums' error): the bound is sum |x||w| times the
    random-walk error of K fp32 additions."""
    x, w = x.double(), w.double()
    y = x @ w.t()
    K = x.shape[1]
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        y = y + bias.double()
        mag = mag + bias.double().abs()
    err = U32 * (2.0 * math.sqrt(K) + 8.0) * mag
    if act == "gelu":
        err = err * 1.13 + 4 * U32 * y.abs()
        y = 0.5 * y * (1.0 + torch.erf(y / math.sqrt(2.0)))
    elif act == "tanh":
        y = torch.tanh(y)
        err = err + 4 * U32
    if res is not None:
        y = y + res.double()
        err = err + U32 * y.abs()
    return y, err


def scores(logits, targets, k, scale=1.0):
    """(logprob, entropy, lse, top, top_id) in fp64 by the header's rules."""
    x = logits.double() * scale
    R, V = x.shape
    raw = logits.double()
    nan = float("nan")
    lp, H, lse = (torch.empty(R, dtype=torch.float64) for _ in range(3))
    top = torch.full((R, k), -math.inf, dtype=torch.float64)
    ids = torch.full((R, k), -1, dtype=torch.int64)
    for r in range(R):
        t = int(targets[r])
        row = x[r]
        if bool(torch.isnan(row).any()) or bool((row == math.inf).any()):
            lse[r] = H[r] = nan
            lp[r] = 0.0 if t < 0 else nan
            top[r] = nan
            continue
        here = row > -math.inf
        if not bool(here.any()):
            lse[r], H[r] = -math.inf, 0.0
            lp[r] = 0.0 if t < 0 else nan if t >= V else -math.inf
            continue
        m = row.max()
        l = (row[here] - m).exp().sum().log()     # apart from m, which may be as large as the type goes
        logp = (row - m) - l
        lse[r], H[r] = m + l, -(logp[here].exp() * logp[here]).sum()
        lp[r] = 0.0 if t < 0 else nan if t >= V else logp[t]
        order = torch.sort(raw[r], descending=True, stable=True).indices[:k]
        n = min(k, int(here.sum()))
        ids[r, :n] = order[:n]
        top[r, :n] = logp[order[:n]]
    return lp, H, lse, top, ids
