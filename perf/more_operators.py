"""The operators of a decoder that answers with drafted tokens, as they are measured.

Four operators, each with its plain form (elementary torch operations in 32
bits, in 64 for angles, sums of logs and borders between tokens, rounded once at the
end), its call through exact_online_amd, and its definition in 64 bits:

* delta: the gated delta rule over given positions.  For every row b, value
  head n (of key head n // (Hv / Hk)) and position t, with a = exp(log_decay),
      u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   S_t = a_t S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t;
  S is the row's state, taken up and left behind (or, held, left as it was: what
  a check of drafted tokens needs).  Positions past a row's length are no positions: o is zero there.
* delta step: the same for one new token of every row; a row's state is
  one slot of a pool.
* rotary: queries and keys normed for each head (divided by their root mean square, times
  weights, or by their length) and turned by their position's angles, in one pass.
* verify: drafted tokens against the target's probabilities.  Draft x_i is kept while u_i q_i(x_i) < p_i(x_i);
  the token after the kept ones is drawn by r from max(p - q, 0) at the first one that is not kept,
  or from p behind the last: the first token whose running sum exceeds r times the whole.  With the target's
  log probability of every token that comes out.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
BYTES = {BF16: 2, F32: 4}
CHUNK = 64   # positions of a chunk of the plain delta form


def listed():
    return [
        # the smallest prompt: a short question on one row, a few narrow heads
        dict(name="delta small", op="delta", B=1, L=77, Hk=4, Hv=4, dk=64, dv=64, dtype=BF16, ragged=False, fresh=True, hold=False),
        # five drafted tokens of every row of a serving batch, run over states that stay as they are until the check
        dict(name="delta drafts", op="delta", B=64, L=5, Hk=16, Hv=32, dk=128, dv=128, dtype=BF16, ragged=False, fresh=False,
             hold=True),
        # a serving batch's ragged prompts that go on from earlier states, value heads sharing queries and keys
        dict(name="delta ragged grouped", op="delta", B=8, L=2048, Hk=16, Hv=32, dk=128, dv=128, dtype=BF16, ragged=True,
             fresh=False, hold=False),
        # the framework's fp32 storage at 1024 channels, an odd length
        dict(name="delta f32", op="delta", B=2, L=4001, Hk=8, Hv=16, dk=64, dv=64, dtype=F32, ragged=False, fresh=True, hold=False),
        # one long document: few heads, 64K positions (the length of the B=8, D=2048 mixer workload)
        dict(name="delta long", op="delta", B=1, L=65536, Hk=16, Hv=16, dk=128, dv=128, dtype=BF16, ragged=False, fresh=True,
             hold=False),
        # one user's next token: latency
        dict(name="delta step one row", op="step", B=1, Hk=16, Hv=16, dk=128, dv=128, dtype=BF16, slots=4),
        # a full serving batch's next tokens, states scattered over a larger pool
        dict(name="delta step batch", op="step", B=200, Hk=16, Hv=32, dk=128, dv=128, dtype=BF16, slots=256),
        # the next token of a few rows, fp32, an odd head size of which a part is turned, lengths of one for the delta rule
        dict(name="rotary tokens", op="rotary", B=7, L=1, Hq=16, Hk=16, d=80, rot=48, norm="l2", pairs="adjacent", dtype=F32, far=True),
        # a prompt of 16K positions, as many as the flagship mixer workload's
        dict(name="rotary prompt", op="rotary", B=1, L=16384, Hq=32, Hk=8, d=128, rot=128, norm="rms", pairs="halves", dtype=BF16,
             far=False),
        # one user's four drafts
        dict(name="verify one row", op="verify", B=1, N=4, V=131072, dtype=F32, drafts="given", ragged=False, pad=0, masked=0.0),
        # a serving batch under a grammar that rules tokens out, an odd vocabulary in padded rows, rows with fewer drafts
        dict(name="verify batch odd", op="verify", B=64, N=5, V=100003, dtype=BF16, drafts="given", ragged=True, pad=61, masked=0.5),
        # drafts looked up in the text so far: certain ones, without probabilities of their own
        dict(name="verify looked up", op="verify", B=96, N=8, V=32768, dtype=BF16, drafts="certain", ragged=False, pad=0, masked=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "step", "rotary", "verify"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("delta", "step"):
        Hk, g = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([1, 1, 2, 3, 4])
        dk, dv = (rng.choice([32, 48, 64, 64, 80, 96, 128, 128, 192, 256]) for _ in range(2))
        if op == "step":
            B = _log(rng, 1, 200)
            return dict(op=op, B=B, Hk=Hk, Hv=Hk * g, dk=dk, dv=dv, dtype=dtype, slots=B + rng.randint(0, 60))
        B = _log(rng, 1, 64)
        L = max(1, min(_log(rng, 1, 65536), 65536 * 16 * 128 * 128 // (B * Hk * g * dk * dv * (4 if dtype == F32 else 1))))
        return dict(op=op, B=B, L=L, Hk=Hk, Hv=Hk * g, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.5,
                    fresh=rng.random() < 0.5, hold=rng.random() < 0.25)
    if op == "rotary":
        d = rng.choice([32, 48, 64, 72, 80, 96, 128, 128, 192, 256])
        Hk, g = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 4, 7])
        B = _log(rng, 1, 64)
        L = max(1, min(_log(rng, 1, 16384), 16384 * 40 * 128 // (B * Hk * (g + 1) * d * (2 if dtype == F32 else 1))))
        return dict(op=op, B=B, L=L, Hq=Hk * g, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2 // 2 * 2, 16, 0]),
                    norm=rng.choice(["rms", "rms", "l2", "none"]), pairs=rng.choice(["halves", "adjacent"]), dtype=dtype,
                    far=rng.random() < 0.5)
    V = _log(rng, 300, 200000)
    N = rng.choice([1, 2, 3, 4, 5, 8])
    B = max(1, min(_log(rng, 1, 256), 64 * 11 * 100003 // ((2 * N + 1) * V) // (2 if dtype == F32 else 1)))
    return dict(op=op, B=B, N=N, V=V, dtype=dtype, drafts=rng.choice(["given", "given", "certain"]), ragged=rng.random() < 0.5,
                pad=rng.choice([0, 0, 7, 64]), masked=rng.choice([0.0, 0.0, 0.5]))


# ------------------------------------------------------------------ inputs
def _stream():
    return torch.cuda.current_stream()


def _lens(c, seed, least):
    """Row lengths on the host, between `least` and L (or N) where they are ragged; the first row is full."""
    most = c["N"] if c["op"] == "verify" else c["L"]
    r = np.random.default_rng([seed, 7])
    n = r.integers(least, most + 1, c["B"]) if c["ragged"] else np.full(c["B"], most)
    n[0] = most
    return n.astype(np.int32)


def _expected(c, least):
    """The expected sum of _lens, for work()."""
    most = c["N"] if c["op"] == "verify" else c["L"]
    return most + (c["B"] - 1) * ((least + most) / 2 if c["ragged"] else most)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=c)
    dt = DTYPES[c["dtype"]]
    if own:
        import exact_online_amd as fi
        io = fi.FI_BF16 if c["dtype"] == BF16 else fi.FI_F32
    if c["op"] in ("delta", "step"):
        B, Hk, Hv, dk, dv = (c[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        L = c.get("L", 1)
        unit = lambda x: torch.nn.functional.normalize(x, dim=-1).to(dt)  # noqa: E731
        # queries and keys have length one, as a model's norms leave them
        s["q"], s["k"] = unit(randn(B, L, Hk, dk)), unit(randn(B, L, Hk, dk))
        s["v"] = randn(B, L, Hv, dv, dtype=dt)
        # a position's decay: a rate of the head (memories of 16 to 4096 positions) times a gate of the position
        rate = torch.exp(-(math.log(16.0) + rand(Hv) * math.log(256.0)))
        s["log_decay"] = -rate * torch.nn.functional.softplus(randn(B, L, Hv))
        s["beta"] = torch.sigmoid(randn(B, L, Hv))
        s["scale"] = 1.0 / math.sqrt(dk)
        s["o"] = torch.empty(B, L, Hv, dv, device="cuda", dtype=dt)
        slots = c.get("slots", B)
        s["state"] = randn(slots, Hv, dk, dv)
        if c["op"] == "step":
            s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)
        else:
            s["lens"] = torch.from_numpy(_lens(c, seed, c["L"] // 4)).cuda() if c["ragged"] else None
        if own:
            s["op"] = fi.DeltaRule(B, L, Hk, Hv, dk, dv, s["scale"], io, stream=_stream())
    elif c["op"] == "rotary":
        B, L, Hq, Hk, d, rot = (c[n] for n in ("B", "L", "Hq", "Hk", "d", "rot"))
        # q and k are parts of one projection's output, as a model has them
        qkv = randn(B, L, (Hq + 2 * Hk) * d, dtype=dt)
        q, k, _ = qkv.split([Hq * d, Hk * d, Hk * d], dim=-1)
        s["q"], s["k"] = q.unflatten(-1, (Hq, d)), k.unflatten(-1, (Hk, d))
        s["qo"], s["ko"] = (torch.empty(B, L, n, d, device="cuda", dtype=dt) for n in (Hq, Hk))
        s["wq"] = s["wk"] = None
        if c["norm"] == "rms":
            s["wq"], s["wk"] = ((1.0 + 0.2 * randn(d)).to(dt) for _ in range(2))
        s["eps"] = 1e-6
        s["freq"] = torch.from_numpy((1e4 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))).astype(np.float32)).cuda()
        # where a row's first position stands: an answer far into a document, or a prompt's beginning
        s["first"] = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda").to(torch.int32) if c["far"] else None
        if own:
            norm = {"none": fi.FI_NORM_NONE, "rms": fi.FI_NORM_RMS, "l2": fi.FI_NORM_L2}[c["norm"]]
            pairs = {"halves": fi.FI_PAIRS_HALVES, "adjacent": fi.FI_PAIRS_ADJACENT}[c["pairs"]]
            s["op"] = fi.Rotary(B, L, Hq, Hk, d, s["freq"], norm, s["eps"], pairs, io, stream=_stream())
    else:
        B, N, V = c["B"], c["N"], c["V"]
        base = randn(B, N + 1, V + c["pad"]) * 3.0
        target = base.to(dt)[..., :V]
        if c["masked"]:
            out = rand(B, N + 1, V) < c["masked"]
            out[..., :64] = False
            target.masked_fill_(out, -math.inf)
        s["target"], s["draft"] = target, None
        # a draft model is near its target; its tokens are drawn from its probabilities
        near = base[:, :N] + randn(B, N, V + c["pad"]) * 0.7
        draft = near.to(dt)[..., :V]
        if c["masked"]:
            draft.masked_fill_(out[:, :N], -math.inf)
        noise = -torch.log(-torch.log(rand(B, N, V).clamp(1e-20, 1.0 - 6e-8)))
        s["tokens"] = (draft.float() + noise).argmax(-1)
        if c["drafts"] == "given":
            s["draft"] = draft
        s["lens"] = torch.from_numpy(_lens(c, seed, 0)).cuda() if c["ragged"] else None
        s["u"], s["r"] = rand(B, N), rand(B)
        s["out"] = torch.empty(B, N + 1, dtype=torch.int64, device="cuda")
        s["kept"], s["logprob"] = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, N + 1, device="cuda")
        if own:
            s["op"] = fi.DraftCheck(B, N, V, io, stream=_stream())
    return s


# ------------------------------------------------------------------ plain forms
def _plain_delta(s):
    """Chunks of CHUNK positions: within a chunk the u of its positions are a triangular system in the keys' products,
    whose inverse is built row by row for all chunks at once; the chunks then follow one another."""
    c = s["case"]
    B, L, Hk, Hv, dk, dv = (c[n] for n in ("B", "L", "Hk", "Hv", "dk", "dv"))
    C = CHUNK
    n = -(-L // C)
    pad = n * C - L
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), L, device="cuda")
    here = torch.arange(n * C, device="cuda")[None, :] < lens[:, None]                  # [B][nC]

    def chunks(x):   # [B][L][h][...] -> [B][Hv][n][C][...]
        x = torch.nn.functional.pad(x.float(), (0, 0) * (x.dim() - 2) + (0, pad))
        x = x.masked_fill(~here.reshape(B, n * C, *(1,) * (x.dim() - 2)), 0.0)
        if x.shape[2] != Hv:
            x = x.repeat_interleave(Hv // Hk, 2)
        return x.transpose(1, 2).unflatten(2, (n, C))
    q, k, v, beta = chunks(s["q"]), chunks(s["k"]), chunks(s["v"]), chunks(s["beta"])
    G = chunks(s["log_decay"]).double().cumsum(-1)                                      # to a position, it included
    i = torch.arange(C, device="cuda")
    lag = G[..., :, None] - G[..., None, :]
    ratio = torch.exp(torch.where(i[:, None] >= i[None, :], lag, -math.inf)).float()
    from_start, to_end, whole = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float(), torch.exp(G[..., -1]).float()
    kt = k.transpose(-1, -2).contiguous()
    A = (k @ kt) * ratio * beta[..., None] * (i[:, None] > i[None, :])
    T = torch.eye(C, device="cuda").expand_as(A).contiguous()
    for r in range(1, C):
        T[..., r, :r] = -(A[..., r, None, :r] @ T[..., :r, :r])[..., 0, :]
    T = T * beta[..., None, :]
    P = (q @ kt) * ratio
    S = s["state"] * (0.0 if c["fresh"] else 1.0)
    o = torch.empty(B, Hv, n, C, dv, device="cuda")
    for m in range(n):
        u = T[:, :, m] @ (v[:, :, m] - from_start[:, :, m, :, None] * (k[:, :, m] @ S))
        o[:, :, m] = from_start[:, :, m, :, None] * (q[:, :, m] @ S) + P[:, :, m] @ u
        S = whole[:, :, m, None, None] * S + kt[:, :, m] @ (u * to_end[:, :, m, :, None])
    o = (o * s["scale"]).reshape(B, Hv, n * C, dv)[:, :, :L].transpose(1, 2)
    s["o"].copy_(o.masked_fill(~here[:, :L, None, None], 0.0))
    if not c["hold"]:
        s["state"].copy_(S)
    return [s["o"], s["state"]]


def _plain_step(s):
    c = s["case"]
    slots = s["slots"].long()
    g = c["Hv"] // c["Hk"]
    q, k = (s[x][:, 0].float().repeat_interleave(g, 1) for x in ("q", "k"))             # [B][Hv][dk]
    S = s["state"][slots] * torch.exp(s["log_decay"][:, 0])[..., None, None]
    u = s["beta"][:, 0, :, None] * (s["v"][:, 0].float() - (k[:, :, None, :] @ S)[:, :, 0])
    S = S + k[..., None] * u[:, :, None, :]
    s["o"].copy_(((q[:, :, None, :] @ S) * s["scale"]).transpose(1, 2))
    s["state"][slots] = S
    return [s["o"], s["state"]]


def _positions(s, B, L):
    t = torch.arange(L, device="cuda")[None, :].expand(B, L)
    return t if s["first"] is None else t + s["first"].long()[:, None]


def _plain_rotary(s):
    c = s["case"]
    rot, d = c["rot"], c["d"]
    angle = _positions(s, c["B"], c["L"]).double()[..., None] * s["freq"].double()     # [B][L][rot / 2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    for x, w, y in ((s["q"], s["wq"], s["qo"]), (s["k"], s["wk"], s["ko"])):
        x = x.float()
        if c["norm"] == "rms":
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        elif c["norm"] == "l2":
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) + s["eps"])
        if w is not None:
            x = x * w.float()
        z = x.clone()
        if c["pairs"] == "halves":
            a, b = slice(0, rot // 2), slice(rot // 2, rot)
        else:
            a, b = slice(0, rot, 2), slice(1, rot, 2)
        z[..., a] = x[..., a] * cos - x[..., b] * sin
        z[..., b] = x[..., b] * cos + x[..., a] * sin
        y.copy_(z)
    return [s["qo"], s["ko"]]


def _plain_verify(s):
    c = s["case"]
    B, N = c["B"], c["N"]

    def probabilities(z):
        z = z.double() - z.double().amax(-1, keepdim=True)
        e = torch.exp(z)
        total = e.sum(-1, keepdim=True)
        return e / total, z - torch.log(total)
    p, logp = probabilities(s["target"])
    q = probabilities(s["draft"])[0] if s["draft"] is not None else None
    x = s["tokens"][..., None]
    px = p[:, :N].gather(-1, x)[..., 0]
    qx = q.gather(-1, x)[..., 0] if q is not None else torch.ones_like(px)
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), N, device="cuda")
    keep = (s["u"].double() * qx < px) & (torch.arange(N, device="cuda")[None, :] < lens[:, None])
    kept = keep.long().cumprod(1).sum(1)
    rows = torch.arange(B, device="cuda")
    w = p[rows, kept]
    stopped, at = kept < lens, kept.clamp(max=N - 1)
    if q is not None:
        rest = (w - q[rows, at]).clamp(min=0.0)
    else:
        rest = w.scatter(1, x[rows, at], 0.0)
    w = torch.where((stopped & (rest.sum(1) > 0.0))[:, None], rest, w)
    run_sum = w.cumsum(1)
    hit = (run_sum > s["r"].double()[:, None] * run_sum[:, -1:]) & (w > 0.0)
    token = hit.to(torch.uint8).argmax(1)
    i = torch.arange(N + 1, device="cuda")[None, :]
    given = torch.nn.functional.pad(s["tokens"], (0, 1))
    s["out"].copy_(torch.where(i < kept[:, None], given, torch.where(i == kept[:, None], token[:, None], -1)))
    s["logprob"].copy_(torch.where(s["out"] >= 0, logp.gather(-1, s["out"].clamp(min=0)[..., None])[..., 0], 0.0))
    s["kept"].copy_(kept)
    return [s["out"], s["kept"], s["logprob"]]


def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        return {"delta": _plain_delta, "step": _plain_step, "rotary": _plain_rotary, "verify": _plain_verify}[op](s)
    if op == "delta":
        s["op"].prompt(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["o"], s["state"], lens=s["lens"], fresh=c["fresh"],
                       hold=c["hold"])
        return [s["o"], s["state"]]
    if op == "step":
        s["op"].step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["o"], s["state"], slots=s["slots"])
        return [s["o"], s["state"]]
    if op == "rotary":
        s["op"].run(s["q"], s["k"], s["qo"], s["ko"], wq=s["wq"], wk=s["wk"], first=s["first"])
        return [s["qo"], s["ko"]]
    s["op"].run(s["target"], s["tokens"], s["u"], s["r"], s["out"], s["kept"], s["logprob"], draft=s["draft"],
                lens=s["lens"])
    return [s["out"], s["kept"], s["logprob"]]


# ------------------------------------------------------------------ work
def work(c):
    n = BYTES[c["dtype"]]
    if c["op"] in ("delta", "step"):
        B, Hk, Hv, dk, dv = (c[x] for x in ("B", "Hk", "Hv", "dk", "dv"))
        T = _expected(c, c["L"] // 4) if c["op"] == "delta" else B
        states = (0 if c.get("fresh") else 1) + (0 if c.get("hold") else 1)
        return dict(bytes=n * T * 2 * (Hk * dk + Hv * dv) + 8 * T * Hv + 4 * B * Hv * dk * dv * states,
                    flops=6 * T * Hv * dk * dv)
    if c["op"] == "rotary":
        heads = c["B"] * c["L"] * (c["Hq"] + c["Hk"])
        return dict(bytes=2 * n * heads * c["d"] + 2 * n * c["d"] + 4 * c["B"], flops=8 * heads * c["d"])
    # the target at every draft and behind the last, the drafts' own where they have any
    rows = _expected(c, 0)
    rows += c["B"] + (rows if c["drafts"] == "given" else 0)
    return dict(bytes=n * rows * c["V"] + c["B"] * (c["N"] * 24 + 28), flops=4 * rows * c["V"])


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_delta(c, s):
    """The recurrence as it stands, position by position, all rows and heads at once."""
    B, Hk, Hv = c["B"], c["Hk"], c["Hv"]
    L, dv = c.get("L", 1), c["dv"]
    slots = s["slots"].long() if "slots" in s else torch.arange(B, device="cuda")
    lens = torch.full((B,), L, device="cuda") if s.get("lens") is None else s["lens"]
    if L * 60e-6 + L * B * Hv * c["dk"] * dv * 100.0 / 3e12 > 15.0:
        return None
    pool = s["state"].double()
    S = pool[slots] if not c.get("fresh") else torch.zeros_like(pool[slots])
    head = torch.arange(Hv, device="cuda") // (Hv // Hk)
    a, beta = s["log_decay"].double().exp(), s["beta"].double()
    o = torch.zeros(B, L, Hv, dv, dtype=torch.float64, device="cuda")
    for t in range(L):
        on = (t < lens).double()[:, None]                                     # no position: nothing changes
        q, k, v = s["q"][:, t, head].double(), s["k"][:, t, head].double(), s["v"][:, t].double()
        S *= (1.0 - on + on * a[:, t])[..., None, None]
        u = (on * beta[:, t])[..., None] * (v - (S * k[..., None]).sum(2))
        S.addcmul_(k[..., None], u[:, :, None, :])
        o[:, t] = (S * q[..., None]).sum(2) * on[..., None]
    if not c.get("hold"):
        pool[slots] = S
    return [s["scale"] * o, pool]


def _exact_rotary(c, s):
    """As products of complex numbers."""
    out = []
    at = _positions(s, c["B"], c["L"]).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[:, :, None, None] * s["freq"].double())
    h = c["rot"] // 2
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        length = x.norm(dim=-1, keepdim=True) ** 2
        if c["norm"] != "none":
            x = x / torch.sqrt((length / c["d"] if c["norm"] == "rms" else length) + s["eps"])
        if w is not None:
            x = x * w.double()
        part, rest = x[..., :2 * h], x[..., 2 * h:]
        part = part.unflatten(-1, (2, h)).transpose(-1, -2) if c["pairs"] == "halves" else part.unflatten(-1, (h, 2))
        z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
        z = z.transpose(-1, -2) if c["pairs"] == "halves" else z
        out.append(torch.cat([z.flatten(-2), rest], -1))
    return out


def _exact_verify(c, s):
    """Row by row, on log probabilities, the running sums searched."""
    B, N = c["B"], c["N"]
    out, count = torch.full((B, N + 1), -1, dtype=torch.int64), torch.zeros(B, dtype=torch.int32)
    logprob = torch.zeros(B, N + 1, dtype=torch.float64)
    u, r, x = s["u"].double().tolist(), s["r"].double().tolist(), s["tokens"].tolist()
    lens = [N] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        p = torch.log_softmax(s["target"][b].double(), -1)
        q = torch.log_softmax(s["draft"][b].double(), -1) if s["draft"] is not None else None
        px = p[torch.arange(N), x[b]].exp().tolist()
        qx = q[torch.arange(N), x[b]].exp().tolist() if q is not None else [1.0] * N
        a = 0
        while a < lens[b] and u[b][a] * qx[a] < px[a]:
            out[b, a] = x[b][a]
            a += 1
        w = p[a].exp()
        if a < lens[b]:
            less = w.clone()
            if q is not None:
                less -= q[a].exp()
            else:
                less[x[b][a]] = 0.0
            less.clamp_(min=0.0)
            w = less if float(less.sum()) > 0.0 else w
        ids = torch.nonzero(w > 0.0)[:, 0]
        sums = w[ids].cumsum(0)
        at = int(torch.searchsorted(sums, sums[-1:] * r[b], right=True))
        out[b, a] = ids[min(at, ids.numel() - 1)]
        count[b] = a
        logprob[b, :a + 1] = p[torch.arange(a + 1), out[b, :a + 1]].cpu()
    return [out.cuda(), count.cuda(), logprob.cuda()]


def exact(c, seed):
    global own
    kept, own = own, False   # inputs alone, no handle
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    return {"delta": _exact_delta, "step": _exact_delta, "rotary": _exact_rotary, "verify": _exact_verify}[c["op"]](c, s)
