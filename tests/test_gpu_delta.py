"""GPU parity of the gated delta rule against its recurrence in 64 bits
(tests/draft_reference.py).

Bounds, set from the arithmetic:
* State, and fp32 outputs: three sums of at most 256 terms lie on each other for a
  position (S^T k, the system of a chunk, the update), each off by sqrt(256) half
  ulps (2^-24) of its terms, which are up to three times their sum: 9 * 16 * 2^-24 = 8.6e-6
  of the norm, bound 1e-5.  Errors of earlier positions pass with the state, which
  |k| = 1 and beta <= 2 do not let grow.
* bf16 outputs: one rounding, of at most half a step, 2^-8 of the value: as |y - x| <= 2^-8 |x|
  for every element, the relative L2 error is <= 2^-8 whatever the values (in the mean 2^-8 / sqrt(3) of a
  power of two, of values with a mean square of 7/3 of it: 2^-9.4; few values can come near the bound).  And an element
  is within 2^-8 of itself and, for what the sums lose before, 2^-12 of the largest.
"""
import math

import pytest

import draft_reference as ref
from fi_harness import log
from op_reference import rel_l2

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)

DT = {"bf16": (torch.bfloat16, fi.FI_BF16), "f32": (torch.float32, fi.FI_F32)}
TOL_STATE, TOL = 1e-5, {"f32": 1e-5, "bf16": 2.0 ** -8}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def stream():
    return torch.cuda.current_stream()


def inputs(seed, B, L, Hk, Hv, dk, dv, dtype, slots=None, memory=(2.0, 500.0)):
    g, dt = gen(seed), DT[dtype][0]
    q, k = (torch.nn.functional.normalize(torch.randn(B, L, Hk, dk, generator=g), dim=-1).to(dt) for _ in range(2))
    v = torch.randn(B, L, Hv, dv, generator=g).to(dt)
    lo, hi = (math.log(x) for x in memory)
    ld = -torch.exp(-(lo + (hi - lo) * torch.rand(B, L, Hv, generator=g)))
    beta = torch.rand(B, L, Hv, generator=g) * 1.2
    return q, k, v, ld, beta, torch.randn(slots or B, Hv, dk, dv, generator=g)


def check_output(o, ro, dtype, what):
    """Every row and head within the bounds."""
    o, ro = o.cpu().double(), ro.double()
    assert bool(torch.isfinite(o).all()), what
    for b in range(o.shape[0]):
        for h in range(o.shape[2]):
            x, y = o[b, :, h], ro[b, :, h]
            e = rel_l2(x, y)
            assert e <= TOL[dtype], (what, b, h, e)
            most = float(y.abs().max()) if y.numel() else 0.0
            if dtype == "bf16":
                assert bool(((x - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -12 * most).all()), (what, b, h)
            else:
                assert bool(((x - y).abs() <= 8 * TOL[dtype] * most).all()), (what, b, h)


def check(x, dtype, lens=None, slots=None, fresh=False, hold=False, dev=None, scale=0.3, mode="prompt", handle=None):
    q, k, v, ld, beta, state = x
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    ro, rs = ref.delta(q, k, v, ld, beta, torch.tensor(scale, dtype=torch.float32).item(), state, lens, slots, fresh, hold)
    d = dev or tuple(t.cuda() for t in (q, k, v, ld, beta))
    o = torch.full((B, L, Hv, dv), 7.0, dtype=q.dtype, device="cuda")
    st = state.cuda()
    log("case delta", mode, dtype, "B", B, "L", L, "H", Hk, Hv, "d", dk, dv, "fresh", fresh, "hold", hold)
    with fi.DeltaRule(*(handle or (B, max(L, 1))), Hk, Hv, dk, dv, scale, DT[dtype][1], stream()) as op:
        ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        if mode == "prompt":
            op.prompt(*d, o, st, lens=ln, slots=sl, fresh=fresh, hold=hold)
        else:
            for t in range(L):
                op.step(*(y[:, t:t + 1] for y in d), o[:, t:t + 1], st, slots=sl)
        torch.cuda.synchronize()
    check_output(o, ro, dtype, "o")
    used = set(range(B)) if slots is None else {s for s in slots if 0 <= s < state.shape[0]}
    for s in range(state.shape[0]):
        if s not in used or hold:
            assert torch.equal(st[s].cpu(), state[s])
        else:
            for n in range(Hv):
                assert rel_l2(st[s, n], rs[s, n]) <= TOL_STATE, (s, n, rel_l2(st[s, n], rs[s, n]))
    return o, st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500])
def test_prompt_lengths(L, dtype):
    check(inputs(L, 2, L, 2, 4, 64, 64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 1, 1), (3, 3, 33, 7), (2, 4, 80, 48), (1, 12, 128, 128), (3, 9, 64, 100),
                                         (2, 2, 256, 256), (5, 5, 192, 40), (2, 20, 16, 136), (1, 2, 130, 250)])
def test_prompt_heads(Hk, Hv, dk, dv, dtype):
    check(inputs(Hv * dk, 2, 150, Hk, Hv, dk, dv, dtype), dtype, fresh=dk == 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [9, 140])
def test_prompt_ragged_and_slots(L, dtype):
    """Rows without positions, of one position, beyond L, out of the pool; NaN
    past every row's end and in the states that no row uses."""
    B = 7
    x = inputs(3, B, L, 2, 4, 64, 96, dtype, slots=9)
    lens = [L, 0, 1, L // 2 + 1, L // 2, -3, 1000]
    slots = [8, 0, 5, 3, -1, 2, 9]
    dev = []
    for y in x[:5]:
        y = y.clone()
        for b in range(B):
            y[b, max(0, min(L, lens[b])):] = float("nan")
        dev.append(y.cuda())
    check(x, dtype, lens=lens, slots=slots, dev=dev)
    check(x, dtype, lens=lens, slots=slots, dev=dev, hold=True)
    slots = [8, 0, 5, 3, 1, 2, 4]
    o, st = check(x, dtype, lens=lens, slots=slots, dev=dev, fresh=True)
    assert float(st[0].abs().max()) == 0.0 and float(o[1].abs().max()) == 0.0   # a fresh row without positions


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [4, 100])
def test_prompt_fresh_ignores_the_state(L, dtype):
    x = inputs(4, 2, L, 2, 2, 64, 64, dtype)
    state = torch.full_like(x[5], float("nan"))
    ro, rs = ref.delta(*x[:5], 1.0, torch.zeros_like(state))
    d = tuple(t.cuda() for t in x[:5])
    with fi.DeltaRule(2, L, 2, 2, 64, 64, 1.0, DT[dtype][1], stream()) as op:
        o, st = torch.empty_like(ro, dtype=x[0].dtype, device="cuda"), state.cuda()
        op.prompt(*d, o, st, fresh=True)
        o2, o3 = torch.empty_like(o), torch.empty_like(o)
        op.prompt(*d, o2, None, fresh=True)      # no state wanted
        st2 = state.cuda()
        op.prompt(*d, o3, st2, fresh=True, hold=True)
        torch.cuda.synchronize()
    check_output(o, ro, dtype, "o")
    assert rel_l2(st, rs) <= TOL_STATE and torch.equal(o, o2) and torch.equal(o, o3)
    assert bool(torch.isnan(st2).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "heads_first", "odd", "shared", "aligned_gap"])
def test_prompt_layouts(layout, dtype):
    B, L, Hk, Hv, dk, dv = 3, 90, 2, 4, 64, 64
    q, k, v, ld, beta, state = inputs(5, B, L, Hk, Hv, dk, dv, dtype)
    gates = torch.stack([ld, beta], -1)          # gates side by side: strides of two
    if layout == "shared":      # one row of keys and values for the whole batch, one gate for every head
        k, v = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
        ld, beta = ld[..., :1].expand(-1, -1, Hv), beta[:, :1].expand(-1, L, -1)
        dev = (q.cuda(), k[:1].contiguous().cuda().expand(B, -1, -1, -1), v[:1].contiguous().cuda().expand(B, -1, -1, -1),
               ld[..., :1].contiguous().cuda().expand(-1, -1, Hv), beta[:, :1].contiguous().cuda().expand(-1, L, -1))
    else:
        if layout == "heads_first":
            dev = tuple(x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (q, k, v))
        else:
            pad = {"fused": 0, "odd": 3, "aligned_gap": 16}[layout]
            whole = torch.cat([x.reshape(B, L, -1) for x in (q, k, v)], -1)
            buf = torch.full((B, L, whole.shape[-1] + pad), float("nan"), dtype=q.dtype, device="cuda")
            start = 1 if layout == "odd" else 0
            buf[..., start:start + whole.shape[-1]] = whole.cuda()
            parts = buf[..., start:start + whole.shape[-1]].split([Hk * dk, Hk * dk, Hv * dv], -1)
            dev = tuple(p.unflatten(-1, (n, d)) for p, n, d in zip(parts, (Hk, Hk, Hv), (dk, dk, dv)))
        g = gates.cuda()
        dev += (g[..., 0], g[..., 1])
    check((q, k, v, ld, beta, state), dtype, dev=dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [3, 70])
def test_prompt_output_views(L, dtype):
    """o as a strided, misaligned view: what lies between stays as it was."""
    B, H, d = 2, 3, 40
    x = inputs(6, B, L, H, H, d, d, dtype)
    ro, _ = ref.delta(*x[:5], 1.0, x[5])
    buf = torch.full((B, L, H, d + 3), 5.0, dtype=x[0].dtype, device="cuda")
    with fi.DeltaRule(B, L, H, H, d, d, 1.0, DT[dtype][1], stream()) as op:
        op.prompt(*(t.cuda() for t in x[:5]), buf[..., 1:d + 1], x[5].cuda())
        torch.cuda.synchronize()
    check_output(buf[..., 1:d + 1], ro, dtype, "o")
    assert bool((buf[..., 0] == 5.0).all()) and bool((buf[..., d + 1:] == 5.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["prompt", "step"])
def test_extreme_gates(mode, dtype):
    """Decays of nothing, of everything (-inf) at some positions, by e^-60, close to one; beta of
    0, 1 (the value is put in the key's place), 2 (mirrored), negative."""
    q, k, v, ld, beta, state = inputs(7, 2, 130, 4, 4, 32, 32, dtype)
    ld[..., 0], ld[..., 1], ld[..., 2] = 0.0, -1e-6, -1e-3
    ld[0, 40, :] = -math.inf
    ld[0, 41, 1] = -math.inf
    ld[1, 60:70, 2] = -60.0
    ld[1, 100, 3] = -1e30
    beta[..., 0] = 1.0
    beta[:, ::3, 1] = 0.0
    beta[..., 2] = 2.0
    beta[..., 3] -= 0.5
    check((q, k, v, ld, beta, state), dtype, mode=mode)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_key_at_every_position(dtype):
    """Keys that are all alike make the system of a chunk as far from the identity as it gets."""
    q, k, v, ld, beta, state = inputs(8, 2, 300, 2, 2, 64, 64, dtype)
    k = k[:, :1].expand(-1, 300, -1, -1).contiguous()
    k[:, 150:, 1] *= -1.0
    check((q, k, v, 0.001 * ld, beta.clamp(max=1.0), state), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_of_other_lengths(dtype):
    """|k|^2 beta up to 1.8, keys of very different sizes, large values and states."""
    q, k, v, ld, beta, state = inputs(9, 2, 200, 2, 2, 64, 32, dtype)
    size = 2.0 ** torch.randint(-6, 7, (2, 200, 2, 1), generator=gen(1))
    k = (k.float() * size).to(k.dtype)
    beta = 1.5 * beta / size[..., 0] ** 2
    check((q, k, (v.float() * 1000).to(v.dtype), ld, beta, state * 1e4), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_memory_of_few_heads(dtype):
    x = inputs(10, 2, 5000, 1, 2, 64, 32, dtype, memory=(2000.0, 8000.0))
    check(x, dtype, lens=[5000, 1027])
    check(inputs(11, 1, 4097, 1, 1, 128, 128, dtype, memory=(1e4, 1e6)), dtype, fresh=True)


@pytest.mark.parametrize("dtype,L", [("bf16", 8400), ("f32", 4200)])
@pytest.mark.parametrize("fresh,hold", [(False, False), (True, True)])
def test_more_chunks_than_are_held_at_a_time(fresh, hold, dtype, L):
    """256 heads of more than 128 chunks: their systems are formed in several runs, states handed from one to the next."""
    x = inputs(20, 4, L, 2, 64, 24, 8, dtype, memory=(100.0, 5000.0))
    check(x, dtype, lens=[L, L - 300, 77, 0], fresh=fresh, hold=hold)


@pytest.mark.parametrize("dtype,L", [("bf16", 300), ("f32", 150)])
def test_many_rows(dtype, L):
    """19200 heads, whose systems of 5 chunks are formed 4 chunks at a time: the same numbers as those of fewer rows."""
    x = inputs(21, 4, L, 2, 32, 24, 8, dtype)
    _, st = check(x, dtype)
    d = [t.cuda().repeat(150, *[1] * (t.dim() - 1)) for t in x]
    o = torch.empty(600, L, 32, 8, dtype=x[2].dtype, device="cuda")
    with fi.DeltaRule(600, L, 2, 32, 24, 8, 0.3, DT[dtype][1], stream()) as op:
        op.prompt(*d[:5], o, d[5])
        torch.cuda.synchronize()
    assert torch.equal(o[:4].repeat(150, 1, 1, 1), o)
    assert torch.equal(st.repeat(150, 1, 1, 1), d[5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_pieces_then_steps(dtype):
    """A prompt in calls of odd lengths and then single steps equals one prompt."""
    B, L, Hk, Hv, d = 2, 203, 2, 4, 64
    x = inputs(12, B, L, Hk, Hv, d, d, dtype)
    ro, rs = ref.delta(*x[:5], 0.125, x[5])
    d_ = [t.cuda() for t in x[:5]]
    o, st = torch.empty(B, L, Hv, d, dtype=x[0].dtype, device="cuda"), x[5].cuda()
    with fi.DeltaRule(B, L, Hk, Hv, d, d, 0.125, DT[dtype][1], stream()) as op:
        for lo, hi in ((0, 77), (77, 80), (80, 190)):
            op.prompt(*(t[:, lo:hi] for t in d_), o[:, lo:hi], st)
        for t in range(190, L):
            op.step(*(y[:, t:t + 1] for y in d_), o[:, t:t + 1], st)
        torch.cuda.synchronize()
    check_output(o, ro, dtype, "o")
    assert rel_l2(st, rs) <= TOL_STATE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", [(1, 1, 1, 1, 1), (3, 16, 16, 128, 128), (5, 2, 8, 64, 96), (2, 1, 9, 33, 130),
                                           (1, 2, 2, 256, 256), (33, 4, 4, 80, 7)])
def test_step(B, Hk, Hv, dk, dv, dtype):
    slots = list(range(B + 2))[::-1][:B]
    check(inputs(B * dk, B, 4, Hk, Hv, dk, dv, dtype, slots=B + 2), dtype, slots=slots, mode="step")


def test_step_rows_out_of_the_pool():
    check(inputs(13, 4, 3, 2, 2, 32, 32, "f32", slots=4), "f32", slots=[3, -1, 4, 0], mode="step")


def test_held_rows_may_share_a_state():
    """Several continuations of one state, none of which changes it."""
    x = list(inputs(14, 3, 6, 2, 4, 64, 64, "bf16", slots=3))
    check(tuple(x), "bf16", slots=[1, 1, 1], hold=True)


def test_a_state_of_many_positions_keeps_its_decay():
    """20000 positions at a = 1 - 1e-5 with nothing added: the state is S_0
    a^20000 (an a rounded to fp32 would be off by up to 20000 * 2^-25 = 6e-4)."""
    d = 16
    state = torch.randn(1, 1, d, d, generator=gen(15))
    z = torch.zeros(1, 20000, 1, d, device="cuda")
    ld, beta = torch.full((1, 20000, 1), -1e-5, device="cuda"), torch.zeros(1, 20000, 1, device="cuda")
    want = state.double() * math.exp(float(ld[0, 0, 0].double()) * 20000)
    for dtype in ("f32", "bf16"):
        zz = z.to(DT[dtype][0])
        o, st = torch.empty_like(zz), state.cuda()
        with fi.DeltaRule(1, 20000, 1, 1, d, d, 1.0, DT[dtype][1], stream()) as op:
            op.prompt(zz, zz, zz, ld, beta, o, st)
            torch.cuda.synchronize()
        assert rel_l2(st, want) <= math.sqrt(20000) * 2 * 2.0 ** -24 + 1e-6


def test_nothing_leaks_from_a_bad_position():
    """A NaN in one row's head stays in that row's head."""
    x = inputs(16, 2, 100, 2, 2, 64, 64, "bf16")
    x[2][0, 70, 1] = float("nan")
    d = tuple(t.cuda() for t in x[:5])
    o, st = torch.empty(2, 100, 2, 64, dtype=torch.bfloat16, device="cuda"), x[5].cuda()
    with fi.DeltaRule(2, 100, 2, 2, 64, 64, 1.0, fi.FI_BF16, stream()) as op:
        op.prompt(*d, o, st)
        torch.cuda.synchronize()
    ro, _ = ref.delta(*x[:5], 1.0, x[5])
    check_output(o[1:], ro[1:], "bf16", "other row")
    check_output(o[:1, :, :1], ro[:1, :, :1], "bf16", "other head")
    assert bool(torch.isnan(o[0, 70:, 1]).all()) and bool(torch.isnan(st[0, 1]).all())
    assert not bool(torch.isnan(o[0, :7, 1]).any())


def test_prompt_of_no_positions_or_rows():
    q, k, v, ld, beta, state = inputs(17, 2, 4, 2, 2, 16, 16, "f32")
    with fi.DeltaRule(2, 4, 2, 2, 16, 16, 1.0, fi.FI_F32, stream()) as op:
        st, o = state.cuda(), torch.empty(2, 4, 2, 16, device="cuda")
        a = [x.cuda() for x in (q, k, v, ld, beta)]
        op.prompt(*[x[:, :0] for x in a], o[:, :0], st)
        assert torch.equal(st.cpu(), state)
        op.prompt(*[x[:0] for x in a], o[:0], st)
        op.step(*[x[:0, :1] for x in a], o[:0, :1], st)
        assert torch.equal(st.cpu(), state)
        op.prompt(*[x[:, :0] for x in a], o[:, :0], st, fresh=True, hold=True)
        assert torch.equal(st.cpu(), state)
        op.prompt(*[x[:, :0] for x in a], o[:, :0], st, fresh=True)
        torch.cuda.synchronize()
        assert float(st.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L", [(1, 2), (1, 65), (1, 300), (1, 2049), (3, 700), (8, 513)])
def test_prompt_on_a_larger_handle(B, L, dtype):
    """A call's plan depends on the call alone: a large handle gives the bits of one made for the call."""
    x = inputs(B * L, B, L, 2, 4, 64, 48, dtype)
    o, st = check(x, dtype, handle=(8, 8192))
    o2, st2 = check(x, dtype)
    assert torch.equal(o, o2) and torch.equal(st, st2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,Hk,Hv", [(2, 1, 2, 2), (2, 5, 2, 4), (1, 1500, 1, 2), (3, 200, 2, 2)])
def test_replays_of_a_graph(B, L, Hk, Hv, dtype):
    """Every replay goes on from the state that the one before left, as calls one after the other do."""
    x = inputs(18, B, L, Hk, Hv, 64, 64, dtype)
    d = [t.cuda() for t in x[:5]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with fi.DeltaRule(B, L, Hk, Hv, 64, 64, 0.5, DT[dtype][1], s) as op, torch.cuda.stream(s):
        eager, states = [], [x[5].cuda()]
        for _ in range(3):
            st = states[-1].clone()
            o = torch.empty(B, L, Hv, 64, dtype=x[0].dtype, device="cuda")
            op.prompt(*d, o, st)
            eager.append(o)
            states.append(st)
        o, st = torch.empty_like(o), x[5].cuda()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            op.prompt(*d, o, st)
        for i in range(3):
            g.replay()
            s.synchronize()
            assert torch.equal(o, eager[i]) and torch.equal(st, states[i + 1]), i
            torch.zeros(1000, device="cuda").sum().item()
    torch.cuda.synchronize()


def test_two_handles_on_two_streams():
    """Calls at once, each on its own handle, stream and state, give what they give alone."""
    x = inputs(19, 2, 1300, 2, 4, 64, 64, "bf16")
    d = [t.cuda() for t in x[:5]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ops = [fi.DeltaRule(2, 1300, 2, 4, 64, 64, 0.5, fi.FI_BF16, s) for s in streams]
    outs = [(torch.empty(2, 1300, 4, 64, dtype=torch.bfloat16, device="cuda"), x[5].cuda()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for op, (o, st) in zip(ops, outs):
            op.prompt(*d, o, st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    with fi.DeltaRule(2, 1300, 2, 4, 64, 64, 0.5, fi.FI_BF16, stream()) as op:
        o, st = torch.empty_like(outs[0][0]), x[5].cuda()
        for _ in range(3):
            op.prompt(*d, o, st)
        torch.cuda.synchronize()
    assert torch.equal(o, outs[0][0]) and torch.equal(st, outs[0][1])
    for op in ops:
        op.close()


def test_refusals():
    q = torch.zeros(2, 4, 2, 8, device="cuda")
    g = torch.zeros(2, 4, 2, device="cuda")
    o, st = torch.empty_like(q), torch.zeros(2, 2, 8, 8, device="cuda")
    with fi.DeltaRule(2, 4, 2, 2, 8, 8, 1.0, fi.FI_F32, stream()) as op:
        def refused(fn, *a, **kw):
            with pytest.raises(fi.FiError) as e:
                fn(*a, **kw)
            assert e.value.status == fi.FI_ERR_INVALID
        refused(op.step, q, q, q, g, g, o, st)                                           # more than one position
        refused(op.prompt, q, q, q, g, g, o, None)                                       # nowhere to begin from
        refused(op.prompt, q, q, q, g, g, o, st[:1])                                     # fewer states than rows
        refused(op.prompt, q, q[..., :4], q, g, g, o, st)                                # another head size
        refused(op.prompt, q, q, q, g[:, :3], g, o, st)                                  # another length
        refused(op.prompt, q, q, q, g, g[..., :1], o, st)                                # a gate too few
        refused(op.prompt, q, q, q, g.double(), g, o, st)
        refused(op.prompt, q, q.transpose(2, 3).contiguous().transpose(2, 3), q, g, g, o, st)   # heads not adjacent
        refused(op.prompt, q.cpu(), q, q, g, g, o, st)
        v = fi.fi_view(q.data_ptr(), 64, 16, 8)
        w = fi.fi_view(g.data_ptr(), 8, 2, 1)
        ok = dict(B=2, L=4, q=v, k=v, v=v, o=fi.fi_view(o.data_ptr(), 64, 16, 8), log_decay=w, beta=w, n_slots=2, state=st.data_ptr())
        assert fi.lib.fi_delta_prompt(op.handle, fi.fi_delta_args(**ok)) == fi.FI_OK
        torch.cuda.synchronize()
