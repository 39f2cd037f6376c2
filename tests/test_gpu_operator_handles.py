"""Calls that are smaller than their handle, on the routes that use its
workspace; calls of several launches in a graph; launches of more workgroups than
are split.  A call's plan depends on the call alone, so a large handle gives
the bits of one made for the call; against the 64-bit forms the bounds of
test_gpu_operators.py hold, here for every row and head by itself."""
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
TOL = {"f32": 5e-6, "bf16": 3 * 2.0 ** -9}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def stream():
    return torch.cuda.current_stream()


def lattn_inputs(seed, B, L, H, Hkv, dk, dv, dtype):
    g, dt = gen(seed), DT[dtype][0]
    q, k, v = (torch.randn(B, L, n, d, generator=g).to(dt) for n, d in ((H, dk), (Hkv, dk), (Hkv, dv)))
    ld = -1.0 / torch.exp(math.log(8.0) + torch.rand(Hkv, generator=g) * math.log(64.0))
    return q, k, v, ld, torch.randn(B, Hkv, dk, dv, generator=g) * 3.0


def run_lattn(handle, x, fresh, scale=0.3):
    """(o, state) of x on a handle of (B, L)."""
    q, k, v, ld, state = x
    B, L, H, dk = q.shape
    Hkv, dv = k.shape[2], v.shape[3]
    o, st = torch.full((B, L, H, dv), 7.0, dtype=q.dtype, device="cuda"), state.cuda()
    io = {d: n for d, n in DT.values()}[q.dtype]
    log("case lattn", "handle", handle, "B", B, "L", L, "H", H, Hkv, "d", dk, dv, q.dtype, "fresh", fresh)
    with fi.LinearAttention(*handle, H, Hkv, dk, dv, ld.cuda(), scale, io, stream()) as op:
        op.prompt(q.cuda(), k.cuda(), v.cuda(), o, st, fresh=fresh)
        torch.cuda.synchronize()
    return o.cpu(), st.cpu()


def every_head(got, want, tol, what):
    """[B, ..., heads, ...] pairs: each row and head within tol of its norm and 8 tol of its largest or rms."""
    for b in range(got.shape[0]):
        for h in range(got.shape[2]):
            g, w = got[b, :, h].double(), want[b, :, h]
            assert ref.rel_l2(g, w) <= tol, (what, b, h)
            assert float((g - w).abs().max()) <= 8 * tol * max(float(w.abs().max()), float(w.square().mean().sqrt())), (what, b, h)


def check_lattn(handle, x, dtype, fresh, scale=0.3):
    q, k, v, ld, state = x
    o, st = run_lattn(handle, x, fresh, scale)
    ro, rs = ref.lattn(q, k, v, ld, torch.tensor(scale, dtype=torch.float32).item(), state, fresh=fresh)
    every_head(o, ro, TOL[dtype], "o")
    every_head(st[:, None], rs[:, None], TOL["f32"], "state")
    return o, st


# ------------------------------------------------------------ smaller calls
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("B,L", [(1, 2), (1, 65), (1, 300), (1, 2049), (3, 700), (8, 513)])
def test_prompt_on_a_larger_handle(B, L, fresh, dtype):
    x = lattn_inputs(B * L, B, L, 6, 2, 64, 48, dtype)
    o, st = check_lattn((8, 8192), x, dtype, fresh)
    o2, st2 = run_lattn((B, L), x, fresh)
    assert torch.equal(o, o2) and torch.equal(st, st2)


@pytest.mark.parametrize("io,N,K,rows", [("bf16", 512, 4160, (64, 200, 33, 17, 5, 4096)), ("f32", 260, 2100, (64, 40, 300, 1)),
                                         ("bf16", 1000, 8200, (129, 256, 20))])
def test_dense_on_a_larger_handle(io, N, K, rows):
    g, dt = gen(N), DT[io][0]
    x, w = torch.randn(max(rows), K, generator=g).to(dt), (torch.randn(N, K, generator=g) / math.sqrt(K)).to(dt)
    bias = torch.randn(N, generator=g).to(dt)
    xd, wd, bd = x.cuda(), w.cuda(), bias.cuda()
    with fi.Dense(4096, N, K, DT[io][1], fi.FI_F32, fi.FI_ACT_TANH, stream()) as op:
        for M in rows:
            y, y2 = (torch.full((M, N), 3.0, device="cuda") for _ in range(2))
            log("case dense", M, N, K, io)
            op.run(xd[:M], wd, y, bias=bd)
            with fi.Dense(M, N, K, DT[io][1], fi.FI_F32, fi.FI_ACT_TANH, stream()) as own:
                own.run(xd[:M], wd, y2, bias=bd)
                torch.cuda.synchronize()
            assert torch.equal(y, y2)
            if M <= 300:
                want, err = ref.dense(x[:M], w, bias, "tanh", None)
                assert bool(((y.cpu().double() - want).abs() <= err + ref.U32 * want.abs() + 1e-30).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_on_a_larger_handle(dtype):
    V, k, g = 50000, 20, gen(5)
    z = (torch.randn(300, V, generator=g) * 3.0).to(DT[dtype][0])
    t = torch.randint(0, V, (300,), generator=g)
    zd, td = z.cuda(), t.cuda()

    def run(op, R):
        out = [torch.full((R,), 9.0, device="cuda") for _ in range(3)]
        out += [torch.full((R, k), 9.0, device="cuda"), torch.full((R, k), 9, dtype=torch.int64, device="cuda")]
        op.run(zd[:R], td[:R], out[0], out[1], out[3], out[4], out[2])
        torch.cuda.synchronize()
        return [x.cpu() for x in out]
    with fi.TokenScores(4096, V, k, DT[dtype][1], 1.0, stream()) as op:
        for R in (1, 7, 300):
            log("case scores", R, V, k, dtype)
            got = run(op, R)
            with fi.TokenScores(R, V, k, DT[dtype][1], 1.0, stream()) as own:
                assert all(torch.equal(a, b) for a, b in zip(got, run(own, R)))
            n = min(R, 7)
            lp, H, lse, top, ids = ref.scores(z[:n], t[:n], k)
            assert torch.equal(got[4][:n], ids)
            for a, b, tol in ((got[0], lp, 8e-6), (got[1], H, 4e-6), (got[2], lse, 4e-6), (got[3], top, 8e-6)):
                assert bool(((a[:n].double() - b).abs() <= tol + 1e-6 * b.abs()).all())


# ------------------------------------------------------------ more workgroups than are split
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,H,Hkv,dk,dv,fresh", [(40, 70, 16, 16, 16, 24, True), (19, 33, 32, 32, 32, 130, False),
                                                    (130, 20, 8, 4, 8, 40, False), (60, 5, 20, 10, 130, 20, True)])
def test_prompt_of_many_rows_and_heads(B, L, H, Hkv, dk, dv, fresh, dtype):
    """Over 512 rows, heads and slices: no segments, no shares of query heads."""
    check_lattn((B, L), lattn_inputs(B, B, L, H, Hkv, dk, dv, dtype), dtype, fresh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["prompt", "step"])
def test_heads_of_very_different_size(mode, dtype):
    """lam = 0, 0.5, 1 - 1e-6 and 1 side by side: the outputs of the first are
    small against those of the last, and each is held to its own size."""
    q, k, v, _, state = lattn_inputs(7, 2, 130, 4, 4, 32, 32, dtype)
    ld = torch.tensor([-math.inf, -math.log(2.0), -1e-6, 0.0])
    if mode == "prompt":
        check_lattn((2, 130), (q, k, v, ld, state), dtype, False)
        return
    ro, rs = ref.lattn(q, k, v, ld, 1.0, state)
    qd, kd, vd, o, st = q.cuda(), k.cuda(), v.cuda(), torch.empty_like(q, device="cuda"), state.cuda()
    with fi.LinearAttention(2, 1, 4, 4, 32, 32, ld.cuda(), 1.0, DT[dtype][1], stream()) as op:
        for t in range(130):
            op.step(*(x[:, t:t + 1] for x in (qd, kd, vd, o)), st)
        torch.cuda.synchronize()
    every_head(o.cpu(), ro, TOL[dtype], "o")
    every_head(st.cpu()[:, None], rs[:, None], TOL["f32"], "state")


# ------------------------------------------------------------ several launches in a graph
def test_calls_of_several_launches_in_a_graph():
    """A prompt in segments, one whose query heads are shared out, a product
    split over K and joined scores, captured on a side stream: every
    replay, between eager runs, equals the eager run bit for bit."""
    g = gen(31)
    H, Hkv, d, L, V, N, K = 8, 2, 64, 1500, 60000, 300, 8192
    q, k, v, ld, state0 = (t.cuda() for t in lattn_inputs(32, 1, L, H, Hkv, d, d, "bf16"))
    x = torch.randn(64, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).bfloat16().cuda()
    z = torch.randn(2, V, generator=g).cuda()
    state, short = state0.clone(), state0.clone()
    o, o2, y = torch.empty_like(q), torch.empty_like(q[:, :40]), torch.empty(64, N, device="cuda")
    H_, top, ids = torch.empty(2, device="cuda"), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, dtype=torch.int64, device="cuda")
    outs = (state, short, o, o2, y, H_, top, ids)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with fi.LinearAttention(1, L, H, Hkv, d, d, ld, 0.2, fi.FI_BF16, side) as mix, \
            fi.Dense(64, N, K, fi.FI_BF16, fi.FI_F32, stream=side) as prod, fi.TokenScores(2, V, 4, fi.FI_F32, stream=side) as sc:
        def run():
            mix.prompt(q, k, v, o, state)
            mix.prompt(q[:, :40], k[:, :40], v[:, :40], o2, short)
            prod.run(x, w, y)
            sc.run(z, entropy=H_, top=top, top_id=ids)
        want = []
        with torch.cuda.stream(side):
            for _ in range(4):
                run()
                side.synchronize()
                want.append([t.clone() for t in outs])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                run()
            state.copy_(state0)
            short.copy_(state0)
            for i in range(4):
                graph.replay()
                side.synchronize()
                for a, b in zip(outs, want[i]):
                    assert torch.equal(a, b), i
                # eager work of the same handles between the replays
                keep = state.clone(), short.clone()
                run()
                side.synchronize()
                state.copy_(keep[0])
                short.copy_(keep[1])
