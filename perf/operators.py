"""The operators of a hybrid decoder around the online mixer, as they are measured.

Four operators, each with its plain form (elementary torch operations in 32
bits, rounded once at the end), its call through exact_online_amd, and its
definition in 64 bits:

* prompt: linear attention with a decay per head over given positions.  For
  every row b, key/value head n and position t (0-indexed, lam = exp(log_decay[n])),
      S_t = lam S_{t-1} + k_t v_t^T,    o_t[h] = scale S_t^T q_t[h],
  h running over the query heads of group n; S is the row's state, taken up and
  left behind.  Positions past a row's length are no positions: o is zero there.
* step: the same recurrence for one new token of every row; a row's state
  is one slot of a pool.
* dense: y = act(x W^T + bias) + residual.
* scores: per row of logits, the log probability of a given token, the
  distribution's entropy, and the k most probable tokens with their log
  probabilities (ties to the lowest index).
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
BYTES = {BF16: 2, F32: 4}
CHUNK = 128   # positions of a chunk of the plain prompt form


def listed():
    return [
        # the smallest call: a short question on one row, a few narrow heads
        dict(name="prompt small", op="prompt", B=1, L=77, H=4, Hkv=4, dk=64, dv=64, dtype=BF16, ragged=False, fresh=True),
        # a serving batch's ragged prompts that go on from earlier states, query heads sharing keys and values
        dict(name="prompt ragged grouped", op="prompt", B=8, L=2048, H=32, Hkv=8, dk=128, dv=128, dtype=BF16, ragged=True,
             fresh=False),
        # the framework's fp32 storage at 1024 channels, an odd length
        dict(name="prompt f32", op="prompt", B=2, L=4001, H=16, Hkv=16, dk=64, dv=64, dtype=F32, ragged=False, fresh=True),
        # one long document: few heads, 64K positions (the length of the B=8, D=2048 mixer workload)
        dict(name="prompt long", op="prompt", B=1, L=65536, H=16, Hkv=16, dk=128, dv=128, dtype=BF16, ragged=False, fresh=True),
        # one user's next token: latency
        dict(name="step one row", op="step", B=1, H=16, Hkv=16, dk=128, dv=128, dtype=BF16, slots=4),
        # a full serving batch's next tokens, states scattered over a larger pool
        dict(name="step batch", op="step", B=200, H=32, Hkv=8, dk=128, dv=128, dtype=BF16, slots=256),
        # the head's product for one token: D=1024 to a vocabulary of 32768, logits kept in fp32
        dict(name="dense one token", op="dense", M=1, N=32768, K=1024, dtype=BF16, out=F32, act="identity", bias=False,
             res=False),
        # a block's first product over a whole prompt (D=1024, L=16K) with bias and GELU
        dict(name="dense prompt", op="dense", M=16384, N=4096, K=1024, dtype=BF16, out=BF16, act="gelu", bias=True, res=False),
        # odd sizes in fp32: the framework's fp32 blocks over a ragged number of rows, with the residual stream added
        dict(name="dense f32 odd", op="dense", M=1777, N=1025, K=999, dtype=F32, out=F32, act="identity", bias=True, res=True),
        # the next token of one row, with the alternatives a sampler or a user sees
        dict(name="scores one row", op="scores", R=1, V=131072, k=20, dtype=F32, masked=0.0, pad=0),
        # scoring a prompt of 4096 tokens
        dict(name="scores prompt", op="scores", R=4096, V=32768, k=5, dtype=BF16, masked=0.0, pad=0),
        # a serving batch under a grammar that rules most tokens out, an odd vocabulary in padded rows
        dict(name="scores masked odd", op="scores", R=333, V=100003, k=8, dtype=BF16, masked=0.9, pad=61),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "dense", "dense", "scores"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("prompt", "step"):
        Hkv, g = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([1, 1, 2, 3, 4])
        dk, dv = (rng.choice([32, 48, 64, 64, 80, 96, 128, 128, 192, 256]) for _ in range(2))
        if op == "step":
            B = _log(rng, 1, 200)
            return dict(op=op, B=B, H=Hkv * g, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, slots=B + rng.randint(0, 60))
        B = _log(rng, 1, 8)
        L = _log(rng, 1, 65536)
        L = max(1, min(L, 65536 * 16 * 512 // (B * Hkv * (dk * (1 + g) + dv * (1 + g)) * (2 if dtype == F32 else 1)),
                       65536 * 16 * 128 // (B * Hkv * g * 128)))
        return dict(op=op, B=B, L=L, H=Hkv * g, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.5,
                    fresh=rng.random() < 0.5)
    if op == "dense":
        most = 16384 * 4096 * 1024
        M, N, K = _log(rng, 1, 16384), _log(rng, 17, 8192), _log(rng, 17, 4096)
        M = max(1, min(M, most // (N * K) // (8 if dtype == F32 else 1)))
        if rng.random() < 0.5:   # models' own widths are rounder than that
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, out=rng.choice([F32, dtype]), act=rng.choice(["identity", "gelu", "tanh"]),
                    bias=rng.random() < 0.6, res=rng.random() < 0.5)
    V = _log(rng, 300, 200000)
    R = max(1, min(_log(rng, 1, 8192), 4096 * 32768 // V // (2 if dtype == F32 else 1)))
    return dict(op=op, R=R, V=V, k=rng.choice([0, 1, 5, 8, 20, 32]), dtype=dtype, masked=rng.choice([0.0, 0.0, 0.5]),
                pad=rng.choice([0, 0, 7, 64]))


# ------------------------------------------------------------------ inputs
def _stream():
    return torch.cuda.current_stream()


def _lens(c, seed):
    """Row lengths on the host: the longest row is full, the others uniform."""
    r = np.random.default_rng([seed, 7])
    n = r.integers(c["L"] // 4, c["L"] + 1, c["B"]) if c["ragged"] else np.full(c["B"], c["L"])
    n[0] = c["L"]
    return n.astype(np.int32)


def _lens_of_case(c):
    """The expected number of positions, for work(): half of the range that _lens draws from, and one full row."""
    return c["L"] + (c["B"] - 1) * (c["L"] * 0.625 if c["ragged"] else c["L"])


def _log_decay(c, gen):
    """lam = exp(-1/tau), tau log-uniform in [64, 8192] positions as the framework's filters."""
    u = torch.rand(c["Hkv"], generator=gen, device="cuda", dtype=torch.float32)
    return -torch.exp(-(math.log(64.0) + u * math.log(8192.0 / 64.0)))


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    s = dict(case=c)
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("prompt", "step"):
        B, H, Hkv, dk, dv = (c[n] for n in ("B", "H", "Hkv", "dk", "dv"))
        L = c.get("L", 1)
        s["log_decay"] = _log_decay(c, g)
        # q, k and v are parts of one projection's output, as a model has them
        qkv = randn(B, L, H * dk + Hkv * (dk + dv), dtype=dt)
        q, k, v = qkv.split([H * dk, Hkv * dk, Hkv * dv], dim=-1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (H, dk)), k.unflatten(-1, (Hkv, dk)), v.unflatten(-1, (Hkv, dv))
        s["scale"] = 1.0 / math.sqrt(dk)
        s["o"] = torch.empty(B, L, H, dv, device="cuda", dtype=dt)
        slots = c.get("slots", B)
        # a state of many positions has a variance of tau / 2
        s["state"] = randn(slots, Hkv, dk, dv) * (-2.0 * s["log_decay"]).rsqrt()[:, None, None]
        if c["op"] == "step":
            s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)
        else:
            s["lens"] = torch.from_numpy(_lens(c, seed)).cuda() if c["ragged"] else None
        if own:
            import exact_online_amd as fi
            s["op"] = fi.LinearAttention(B, L, H, Hkv, dk, dv, s["log_decay"], s["scale"],
                                         fi.FI_BF16 if c["dtype"] == BF16 else fi.FI_F32, stream=_stream())
    elif c["op"] == "dense":
        M, N, K = c["M"], c["N"], c["K"]
        to = DTYPES[c["out"]]
        s["x"] = randn(M, K, dtype=dt)
        s["w"] = (randn(N, K) / math.sqrt(K)).to(dt)
        s["bias"] = (randn(N) * 0.1).to(dt) if c["bias"] else None
        s["res"] = randn(M, N, dtype=to) if c["res"] else None
        s["y"] = torch.empty(M, N, device="cuda", dtype=to)
        if own:
            import exact_online_amd as fi
            name = {BF16: fi.FI_BF16, F32: fi.FI_F32}
            act = {"identity": fi.FI_ACT_IDENTITY, "gelu": fi.FI_ACT_GELU, "tanh": fi.FI_ACT_TANH}[c["act"]]
            s["op"] = fi.Dense(M, N, K, name[c["dtype"]], name[c["out"]], act, stream=_stream())
    else:
        R, V, k = c["R"], c["V"], c["k"]
        logits = (randn(R, V + c["pad"]) * 3.0).to(dt)[:, :V]
        s["targets"] = torch.randint(0, V, (R,), generator=g, device="cuda")
        if c["masked"]:
            keep = torch.rand(R, V, generator=g, device="cuda") >= c["masked"]
            keep.scatter_(1, s["targets"][:, None], True)   # the token that was taken was allowed
            keep[:, :64] = True
            logits.masked_fill_(~keep, -math.inf)
        s["logits"] = logits
        s["logprob"], s["entropy"] = (torch.empty(R, device="cuda") for _ in range(2))
        s["top"] = torch.empty(R, k, device="cuda")
        s["top_id"] = torch.empty(R, k, device="cuda", dtype=torch.int64)
        if own:
            import exact_online_amd as fi
            s["op"] = fi.TokenScores(R, V, k, fi.FI_BF16 if c["dtype"] == BF16 else fi.FI_F32, stream=_stream())
    return s


# ------------------------------------------------------------------ plain forms
def _plain_prompt(s):
    """Chunks of CHUNK positions: the part of a chunk's own positions as a masked product, that of earlier ones through
    the chunks' states, which a product with the decays between chunks gives."""
    c = s["case"]
    B, L, H, Hkv, dk, dv = (c[n] for n in ("B", "L", "H", "Hkv", "dk", "dv"))
    G, C = H // Hkv, CHUNK
    n = -(-L // C)
    pad = n * C - L
    ld = s["log_decay"]
    t = torch.arange(n * C, device="cuda")
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), L, device="cuda")
    here = t[None, :] < lens[:, None]                                              # [B][nC]
    heads_first = lambda x: torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad)).transpose(1, 2)  # noqa: E731
    q = heads_first(s["q"]).masked_fill_(~here[:, None, :, None], 0.0)
    k = heads_first(s["k"]).masked_fill_(~here[:, None, :, None], 0.0).reshape(B, Hkv, n, C, dk)
    v = heads_first(s["v"]).masked_fill_(~here[:, None, :, None], 0.0).reshape(B, Hkv, n, C, dv)
    q = q.reshape(B, Hkv, G, n, C, dk).transpose(2, 3).reshape(B, Hkv, n, G * C, dk)   # a group's rows beside each other
    i = torch.arange(C, device="cuda")
    lag = i[:, None] - i[None, :]
    within = torch.exp(ld[:, None, None] * lag.clamp(min=0)) * (lag >= 0)              # [Hkv][C][C]
    p = (q @ k.transpose(-1, -2).contiguous()) * within.repeat(1, G, 1)[:, None]
    o = p @ v
    # U[c]: a chunk's own state at its end; E[c]: the state before chunk c
    to_end = torch.exp(ld[:, None] * (C - 1 - i))                                      # [Hkv][C]
    U = (k * to_end[:, None, :, None]).transpose(-1, -2).contiguous() @ v              # [B][Hkv][n][dk][dv]
    m = torch.arange(n, device="cuda")
    ago = m[:, None] - 1 - m[None, :]
    between = torch.exp(ld[:, None, None] * (C * ago.clamp(min=0))) * (ago >= 0)       # [Hkv][n][n]
    E = (between @ U.flatten(-2)).unflatten(-1, (dk, dv))
    if not c["fresh"]:
        E = E + torch.exp(ld[:, None] * (C * m))[..., None, None] * s["state"][:, :, None]
    from_start = torch.exp(ld[:, None] * (i + 1)).repeat(1, G)                         # [Hkv][G C]
    o = (o + (q * from_start[:, None, :, None]) @ E) * s["scale"]
    o = o.reshape(B, Hkv, n, G, C, dv).permute(0, 2, 4, 1, 3, 5).reshape(B, n * C, H, dv)[:, :L]
    # the state after the last position of each row: of its last chunk, less the decay of the places behind its end
    last = ((lens - 1).clamp(min=0) // C).long()
    at = torch.arange(B, device="cuda")
    whole = torch.exp(ld * C)[None, :, None, None] * E[at, :, last] + U[at, :, last]
    over = (last + 1) * C - lens
    state = whole * torch.exp(-ld[None, :] * over[:, None])[..., None, None]
    s["o"].copy_(o)
    s["state"].copy_(state)
    return [s["o"], s["state"]]


def _plain_step(s):
    c = s["case"]
    slots = s["slots"].long()
    B, H, Hkv, dk, dv = (c[n] for n in ("B", "H", "Hkv", "dk", "dv"))
    S = s["state"][slots] * torch.exp(s["log_decay"])[:, None, None]
    S = S + s["k"].float().reshape(B, Hkv, dk, 1) * s["v"].float().reshape(B, Hkv, 1, dv)
    o = (s["q"].float().reshape(B, Hkv, H // Hkv, dk) @ S) * s["scale"]
    s["state"][slots] = S
    s["o"].copy_(o.reshape(B, 1, H, dv))
    return [s["o"], s["state"]]


def _plain_dense(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    act = s["case"]["act"]
    if act == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif act == "tanh":
        y = torch.tanh(y)
    if s["res"] is not None:
        y = y + s["res"].float()
    s["y"].copy_(y)
    return s["y"]


def _plain_scores(s):
    c = s["case"]
    x = s["logits"].float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    total = e.sum(1, keepdim=True)
    lp = x - (x.amax(1, keepdim=True) + torch.log(total))
    p = e / total
    entropy = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    out = [lp.gather(1, s["targets"][:, None])[:, 0], entropy]
    if c["k"]:
        # ties to the lowest index: the order of the values' bits, then that of the places from the back
        bits = (x + 0.0).view(torch.int32).to(torch.int64)
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        places = torch.arange(c["V"] - 1, -1, -1, device="cuda")
        key = torch.topk((order << 32) + places, c["k"], dim=1).values
        ids = c["V"] - 1 - (key & 0xFFFFFFFF)
        out += [lp.gather(1, ids), ids]
    return out


def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        return {"prompt": _plain_prompt, "step": _plain_step, "dense": _plain_dense, "scores": _plain_scores}[op](s)
    if op == "prompt":
        s["op"].prompt(s["q"], s["k"], s["v"], s["o"], s["state"], lens=s["lens"], fresh=c["fresh"])
        return [s["o"], s["state"]]
    if op == "step":
        s["op"].step(s["q"], s["k"], s["v"], s["o"], s["state"], slots=s["slots"])
        return [s["o"], s["state"]]
    if op == "dense":
        s["op"].run(s["x"], s["w"], s["y"], bias=s["bias"], res=s["res"])
        return s["y"]
    s["op"].run(s["logits"], s["targets"], s["logprob"], s["entropy"], s["top"], s["top_id"])
    return [s["logprob"], s["entropy"]] + ([s["top"], s["top_id"]] if c["k"] else [])


# ------------------------------------------------------------------ work
def work(c):
    n = BYTES[c["dtype"]]
    if c["op"] in ("prompt", "step"):
        B, H, Hkv, dk, dv = (c[x] for x in ("B", "H", "Hkv", "dk", "dv"))
        T = _lens_of_case(c) if c["op"] == "prompt" else B
        read = 0 if c.get("fresh") else 1
        return dict(bytes=n * T * (H * (dk + dv) + Hkv * (dk + dv)) + 4 * B * Hkv * dk * dv * (read + 1) + 4 * Hkv,
                    flops=2 * T * dk * dv * (H + Hkv))
    if c["op"] == "dense":
        M, N, K = c["M"], c["N"], c["K"]
        m = BYTES[c["out"]]
        return dict(bytes=n * (M * K + N * K + N * c["bias"]) + m * M * N * (1 + c["res"]), flops=2 * M * N * K)
    R, V, k = c["R"], c["V"], c["k"]
    return dict(bytes=n * R * V + R * (8 + 4 + 4) + R * k * (4 + 8), flops=6 * R * V)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_prompt(c, s):
    """o_i = scale (lam^{i+1} S_0^T q_i + sum_{j<=i} lam^{i-j} (q_i . k_j) v_j), row by row and head by head, over
    blocks of queries (and blocks of keys no further back than lam reaches 2^-100)."""
    B, L, H, Hkv, dk, dv = (c[n] for n in ("B", "L", "H", "Hkv", "dk", "dv"))
    G = H // Hkv
    o = torch.zeros(B, L, H, dv, dtype=torch.float64, device="cuda")
    state = s["state"].double() * (0.0 if c["fresh"] else 1.0)
    if B * Hkv * G * (float(L) ** 2) * (dk + dv) > 2e14:
        return None
    for b in range(B):
        n = L if s["lens"] is None else int(s["lens"][b])
        for m in range(Hkv):
            ld = s["log_decay"][m].double()
            reach = int(100.0 / float(-ld))
            k, v = s["k"][b, :n, m].double(), s["v"][b, :n, m].double()
            S0 = state[b, m].clone()
            for i0 in range(0, n, 1024):
                i1, j0 = min(n, i0 + 1024), max(0, i0 - reach)
                lag = torch.arange(i0, i1, device="cuda")[:, None] - torch.arange(j0, i1, device="cuda")[None, :]
                w = torch.where(lag >= 0, torch.exp(ld * lag), 0.0)
                first = torch.exp(ld * torch.arange(i0 + 1, i1 + 1, device="cuda"))[:, None]
                for g in range(G):
                    q = s["q"][b, i0:i1, m * G + g].double()
                    a = torch.mm(q, k[j0:i1].t().contiguous()) * w
                    o[b, i0:i1, m * G + g] = s["scale"] * (torch.mm(a, v[j0:i1]) + first * torch.mm(q, S0))
            w = torch.exp(ld * torch.arange(n - 1, -1, -1, device="cuda"))[:, None]
            state[b, m] = torch.exp(ld * n) * S0 + torch.mm((k * w).t().contiguous(), v)
    return [o, state]


def _exact_step(c, s):
    B, H, Hkv, dk, dv = (c[n] for n in ("B", "H", "Hkv", "dk", "dv"))
    G = H // Hkv
    state = s["state"].double()
    o = torch.zeros(B, 1, H, dv, dtype=torch.float64, device="cuda")
    lam = torch.exp(s["log_decay"].double())
    for b in range(B):
        at = int(s["slots"][b])
        for m in range(Hkv):
            S = lam[m] * state[at, m] + torch.outer(s["k"][b, 0, m].double(), s["v"][b, 0, m].double())
            state[at, m] = S
            o[b, 0, m * G:(m + 1) * G] = s["scale"] * torch.mm(s["q"][b, 0, m * G:(m + 1) * G].double(), S)
    return [o, state]


def _exact_dense(c, s):
    y = torch.mm(s["x"].double(), s["w"].double().t().contiguous())
    if s["bias"] is not None:
        y += s["bias"].double()[None, :]
    if c["act"] == "gelu":
        y *= torch.special.ndtr(y)
    elif c["act"] == "tanh":
        y.tanh_()
    return y if s["res"] is None else y + s["res"].double()


def _exact_scores(c, s):
    logprob, entropy, top = [], [], []
    for r in range(0, c["R"], 256):
        x = s["logits"][r:r + 256].double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        logprob.append(lp.gather(1, s["targets"][r:r + 256, None])[:, 0])
        entropy.append(-torch.special.xlogy(lp.exp(), lp.exp()).sum(1))
        if c["k"]:
            top.append(lp.sort(1, descending=True).values[:, :c["k"]])
    return [torch.cat(logprob), torch.cat(entropy)] + ([torch.cat(top), None] if c["k"] else [])


def exact(c, seed):
    global own
    kept, own = own, False   # inputs alone, no handle
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    return {"prompt": _exact_prompt, "step": _exact_step, "dense": _exact_dense, "scores": _exact_scores}[c["op"]](c, s)
