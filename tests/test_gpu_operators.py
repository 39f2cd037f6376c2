"""GPU parity of the operators around the mixers against their plain forms in
64 bits (tests/op_reference.py).

Bounds, set from the arithmetic:
* fp32 sums of n terms err by about sqrt(n) half ulps (2^-24) of the terms'
  size, chained over at most four such sums (n <= 256 each, 64 to 1024
  positions between roundings): relative L2 error of linear attention's state
  and of its fp32 output <= 5e-6.
* a bf16 output is rounded once, and the chunked form rounds the scores within
  a chunk and the entry state to bf16 operands (each a part of the output); a
  rounding to bf16 errs by 2^-8 at most and by about 2^-9 in the mean square:
  relative L2 error <= 3 * 2^-9 < 6e-3.  Values are compared
  element by element too, against 8 times that of the row's largest.
* dense products: per element, from sum |x||w| (op_reference.dense), and one
  rounding to the output's type.
* scores: 2^t is off by |t| 2^-23, so log probabilities by 1e-6 (8 + |lp|) and
  entropies by 1e-6 (4 + H).
"""
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
TOL_F32, TOL_BF16 = 5e-6, 3 * 2.0 ** -9


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def stream():
    return torch.cuda.current_stream()


# ------------------------------------------------------------ linear attention
def lattn_inputs(seed, B, L, H, Hkv, dk, dv, dtype, slots=None):
    g, dt = gen(seed), DT[dtype][0]
    q = torch.randn(B, L, H, dk, generator=g).to(dt)
    k = torch.randn(B, L, Hkv, dk, generator=g).to(dt)
    v = torch.randn(B, L, Hkv, dv, generator=g).to(dt)
    ld = -torch.exp(-torch.rand(Hkv, generator=g) * 7.0)      # memories of 1 to 1000 positions
    state = torch.randn(slots or B, Hkv, dk, dv, generator=g) * 3.0
    return q, k, v, ld, state


def close(o, ro, dtype, what):
    o, ro = o.cpu().double(), ro.double()
    assert torch.isfinite(o).all(), what
    tol = TOL_F32 if dtype == "f32" else TOL_BF16
    e = ref.rel_l2(o, ro)
    worst = ((o - ro).abs().amax(-1) / ro.abs().amax(-1).clamp(min=1e-30)).max() if o.numel() else 0.0
    log(what, "rel l2 %.3g, worst %.3g" % (e, worst))
    assert e <= tol, what
    # a row's largest value may be small against the terms that made it
    rms = float(ro.square().mean().sqrt()) if ro.numel() else 1.0
    assert (o - ro).abs().max() <= 8 * tol * max(float(ro.abs().max()), rms) if o.numel() else True, what


def check_lattn(inputs, dtype, lens=None, slots=None, fresh=False, dev=None, scale=0.3, mode="prompt"):
    q, k, v, ld, state = inputs
    B, L, H, dk = q.shape
    Hkv, dv = k.shape[2], v.shape[3]
    ro, rs = ref.lattn(q, k, v, ld, torch.tensor(scale, dtype=torch.float32).item(), state, lens, slots, fresh)
    dq, dkk, dvv = dev or (q.cuda(), k.cuda(), v.cuda())
    o = torch.full((B, L, H, dv), 7.0, dtype=q.dtype, device="cuda")
    st = state.cuda()
    log("case lattn", mode, dtype, "B", B, "L", L, "H", H, Hkv, "d", dk, dv, "fresh", fresh)
    with fi.LinearAttention(B, max(L, 1), H, Hkv, dk, dv, ld.cuda(), scale, DT[dtype][1], stream()) as op:
        ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        if mode == "prompt":
            op.prompt(dq, dkk, dvv, o, st, lens=ln, slots=sl, fresh=fresh)
        else:
            for t in range(L):
                op.step(dq[:, t:t + 1], dkk[:, t:t + 1], dvv[:, t:t + 1], o[:, t:t + 1], st, slots=sl)
        torch.cuda.synchronize()
    close(o, ro, dtype, "o")
    # states that no row of the call uses are as they were; the others within the fp32 bound
    used = set(range(B)) if slots is None else {s for s in slots if 0 <= s < state.shape[0]}
    for s in range(state.shape[0]):
        if s not in used:
            assert torch.equal(st[s].cpu(), state[s])
    assert ref.rel_l2(st, rs) <= TOL_F32
    return o, st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500])
def test_prompt_lengths(L, dtype):
    check_lattn(lattn_inputs(L, 2, L, 4, 2, 64, 64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,dk,dv", [(1, 1, 1, 1), (3, 3, 33, 7), (4, 2, 80, 48), (12, 1, 128, 128), (9, 3, 64, 100),
                                         (2, 2, 256, 256), (5, 5, 192, 40), (20, 2, 16, 136), (2, 1, 130, 250)])
def test_prompt_heads(H, Hkv, dk, dv, dtype):
    check_lattn(lattn_inputs(H * dk, 2, 150, H, Hkv, dk, dv, dtype), dtype, fresh=dk == 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_ragged_and_slots(dtype):
    """Rows without positions, of one position, beyond L, out of the pool; NaN
    past every row's end and in the states that no row uses."""
    B, L = 7, 140
    q, k, v, ld, state = lattn_inputs(3, B, L, 4, 2, 64, 96, dtype, slots=9)
    lens = [140, 0, 1, 65, 64, -3, 1000]
    slots = [8, 0, 5, 3, -1, 2, 9]
    dev = []
    for x in (q, k, v):
        y = x.clone()
        for b in range(B):
            y[b, max(0, min(L, lens[b])):] = float("nan")
        dev.append(y.cuda())
    check_lattn((q, k, v, ld, state), dtype, lens=lens, slots=slots, dev=dev)
    slots = [8, 0, 5, 3, 1, 2, 4]
    o, st = check_lattn((q, k, v, ld, state), dtype, lens=lens, slots=slots, dev=dev, fresh=True)
    assert float(st[0].abs().max()) == 0.0 and float(o[1].abs().max()) == 0.0   # a fresh row without positions


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_fresh_ignores_the_state(dtype):
    x = lattn_inputs(4, 2, 100, 2, 2, 64, 64, dtype)
    state = torch.full_like(x[4], float("nan"))
    q, k, v, ld, _ = x
    ro, rs = ref.lattn(q, k, v, ld, 1.0, torch.zeros_like(state))
    with fi.LinearAttention(2, 100, 2, 2, 64, 64, ld.cuda(), 1.0, DT[dtype][1], stream()) as op:
        o, st = torch.empty_like(ro, dtype=q.dtype, device="cuda"), state.cuda()
        op.prompt(q.cuda(), k.cuda(), v.cuda(), o, st, fresh=True)
        o2 = torch.empty_like(o)
        op.prompt(q.cuda(), k.cuda(), v.cuda(), o2, None, fresh=True)      # no state wanted
        torch.cuda.synchronize()
    close(o, ro, dtype, "o")
    assert ref.rel_l2(st, rs) <= TOL_F32 and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "heads_first", "odd", "shared", "aligned_gap"])
def test_prompt_layouts(layout, dtype):
    B, L, H, Hkv, dk, dv = 3, 90, 4, 2, 64, 64
    q, k, v, ld, state = lattn_inputs(5, B, L, H, Hkv, dk, dv, dtype)
    if layout == "shared":      # one row of keys and values for the whole batch
        k, v = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
        dev = (q.cuda(), k[:1].contiguous().cuda().expand(B, -1, -1, -1), v[:1].contiguous().cuda().expand(B, -1, -1, -1))
    elif layout == "heads_first":
        dev = tuple(x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (q, k, v))
    else:
        pad = {"fused": 0, "odd": 3, "aligned_gap": 16}[layout]
        whole = torch.cat([x.reshape(B, L, -1) for x in (q, k, v)], -1)
        buf = torch.full((B, L, whole.shape[-1] + pad), float("nan"), dtype=q.dtype, device="cuda")
        start = 1 if layout == "odd" else 0
        buf[..., start:start + whole.shape[-1]] = whole.cuda()
        parts = buf[..., start:start + whole.shape[-1]].split([H * dk, Hkv * dk, Hkv * dv], -1)
        dev = tuple(p.unflatten(-1, (n, d)) for p, n, d in zip(parts, (H, Hkv, Hkv), (dk, dk, dv)))
    check_lattn((q, k, v, ld, state), dtype, dev=dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_output_views(dtype):
    """o as a strided, misaligned view: what lies between stays as it was."""
    B, L, H, d = 2, 70, 3, 40
    q, k, v, ld, state = lattn_inputs(6, B, L, H, H, d, d, dtype)
    ro, _ = ref.lattn(q, k, v, ld, 1.0, state)
    buf = torch.full((B, L, H, d + 3), 5.0, dtype=q.dtype, device="cuda")
    with fi.LinearAttention(B, L, H, H, d, d, ld.cuda(), 1.0, DT[dtype][1], stream()) as op:
        op.prompt(q.cuda(), k.cuda(), v.cuda(), buf[..., 1:d + 1], state.cuda())
        torch.cuda.synchronize()
    close(buf[..., 1:d + 1], ro, dtype, "o")
    assert bool((buf[..., 0] == 5.0).all()) and bool((buf[..., d + 1:] == 5.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["prompt", "step"])
def test_extreme_decays(mode, dtype):
    """lam = 0 (only a position's own key and value), 1 (nothing is lost),
    0.5 per position, and close to 1."""
    q, k, v, _, state = lattn_inputs(7, 2, 130, 4, 4, 32, 32, dtype)
    ld = torch.tensor([-math.inf, 0.0, -math.log(2.0), -1e-6])
    check_lattn((q, k, v, ld, state), dtype, mode=mode)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_memory_of_few_heads(dtype):
    """The split over positions: few heads, many chunks, long and short rows."""
    q, k, v, _, state = lattn_inputs(8, 2, 5000, 2, 1, 64, 32, dtype)
    ld = torch.tensor([-1.0 / 4096])
    check_lattn((q, k, v, ld, state), dtype, lens=[5000, 1027])
    q, k, v, ld, state = lattn_inputs(9, 1, 4097, 1, 1, 128, 128, dtype)
    check_lattn((q, k, v, ld * 0.001, state), dtype, fresh=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_pieces_then_steps(dtype):
    """A prompt in two calls of odd lengths and then single steps equals one prompt."""
    B, L, H, Hkv, d = 2, 203, 4, 2, 64
    q, k, v, ld, state = lattn_inputs(10, B, L, H, Hkv, d, d, dtype)
    ro, rs = ref.lattn(q, k, v, ld, 0.125, state)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    o, st = torch.empty(B, L, H, d, dtype=q.dtype, device="cuda"), state.cuda()
    with fi.LinearAttention(B, L, H, Hkv, d, d, ld.cuda(), 0.125, DT[dtype][1], stream()) as op:
        for lo, hi in ((0, 77), (77, 190)):
            op.prompt(q[:, lo:hi], k[:, lo:hi], v[:, lo:hi], o[:, lo:hi], st)
        for t in range(190, L):
            op.step(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], o[:, t:t + 1], st)
        torch.cuda.synchronize()
    close(o, ro, dtype, "o")
    assert ref.rel_l2(st, rs) <= TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hkv,dk,dv", [(1, 1, 1, 1, 1), (3, 16, 16, 128, 128), (5, 8, 2, 64, 96), (2, 9, 1, 33, 130),
                                           (1, 2, 2, 256, 256), (33, 4, 4, 80, 7)])
def test_step(B, H, Hkv, dk, dv, dtype):
    slots = list(range(B + 2))[::-1][:B]
    x = lattn_inputs(B * dk, B, 4, H, Hkv, dk, dv, dtype, slots=B + 2)
    check_lattn(x, dtype, slots=slots, mode="step")


def test_step_rows_out_of_the_pool():
    x = lattn_inputs(11, 4, 3, 2, 2, 32, 32, "f32", slots=4)
    check_lattn(x, "f32", slots=[3, -1, 4, 0], mode="step")


def test_a_state_of_many_steps_keeps_its_decay():
    """20000 steps at lam = 1 - 1e-5 with nothing added: the state is S_0
    lam^20000 (a lam rounded to fp32 would be off by up to 20000 * 2^-25 =
    6e-4)."""
    d = 16
    state = torch.randn(1, 1, d, d, generator=gen(12))
    ld = torch.tensor([-1e-5])
    z = torch.zeros(1, 1, 1, d, device="cuda")
    o, st = torch.empty_like(z), state.cuda()
    with fi.LinearAttention(1, 1, 1, 1, d, d, ld.cuda(), 1.0, fi.FI_F32, stream()) as op:
        for _ in range(20000):
            op.step(z, z, z, o, st)
        torch.cuda.synchronize()
    want = state.double() * math.exp(float(ld[0].double()) * 20000)
    assert ref.rel_l2(st, want) <= math.sqrt(20000) * 2 * ref.U32 + 1e-6


def test_prompt_of_no_positions_or_rows():
    q, k, v, ld, state = lattn_inputs(13, 2, 4, 2, 2, 16, 16, "f32")
    with fi.LinearAttention(2, 4, 2, 2, 16, 16, ld.cuda(), 1.0, fi.FI_F32, stream()) as op:
        st, o = state.cuda(), torch.empty(2, 4, 2, 16, device="cuda")
        a = [x.cuda() for x in (q, k, v)]
        op.prompt(*[x[:, :0] for x in a], o[:, :0], st)
        assert torch.equal(st.cpu(), state)
        op.prompt(*[x[:0] for x in a], o[:0], st)
        op.step(*[x[:0, :1] for x in a], o[:0, :1], st)
        assert torch.equal(st.cpu(), state)
        op.prompt(*[x[:, :0] for x in a], o[:, :0], st, fresh=True)
        torch.cuda.synchronize()
        assert float(st.abs().max()) == 0.0


def test_lattn_refusals():
    ld = torch.tensor([-0.1, -0.2], device="cuda")
    for bad in ([0.1, -1.0], [float("nan"), -1.0], [-1.0, float("inf")]):
        with pytest.raises(fi.FiError) as e:
            fi.LinearAttention(1, 4, 2, 2, 8, 8, torch.tensor(bad, device="cuda"), 1.0, fi.FI_F32, stream())
        assert e.value.status == fi.FI_ERR_INVALID
    q = torch.zeros(2, 4, 2, 8, device="cuda")
    o, st = torch.empty_like(q), torch.zeros(2, 2, 8, 8, device="cuda")
    with fi.LinearAttention(2, 4, 2, 2, 8, 8, ld, 1.0, fi.FI_F32, stream()) as op:
        def refused(fn, *a, **kw):
            with pytest.raises(fi.FiError) as e:
                fn(*a, **kw)
            assert e.value.status == fi.FI_ERR_INVALID
        refused(op.step, q, q, q, o, st)                                           # more than one position
        refused(op.prompt, q, q, q, o, None)                                       # nowhere to begin from
        refused(op.prompt, q, q, q, o, st[:1])                                     # fewer states than rows
        refused(op.prompt, q, q[..., :4], q, o, st)                                # another head size
        refused(op.prompt, q, q[:, :3], q, o, st)                                  # another length
        refused(op.prompt, q, q.transpose(2, 3).contiguous().transpose(2, 3), q, o, st)   # heads not adjacent
        refused(op.prompt, torch.zeros(3, 4, 2, 8, device="cuda"), q, q, o, st)
        big = torch.zeros(2, 5, 2, 8, device="cuda")
        refused(op.prompt, big, big, big, torch.empty_like(big), st)               # beyond the config's L
        v = fi.fi_view(q.data_ptr(), 64, 16, 8)
        ok = dict(B=2, L=4, q=v, k=v, v=v, o=fi.fi_view(o.data_ptr(), 64, 16, 8), n_slots=2, state=st.data_ptr())
        for kw in (dict(B=3), dict(B=-1), dict(L=-1), dict(q=fi.fi_view(0, 64, 16, 8)), dict(n_slots=1), dict(n_slots=-1),
                   dict(q=fi.fi_view(q.data_ptr() + 2, 64, 16, 8)), dict(state=0), dict(state=st.data_ptr() + 4),
                   dict(lens=q.data_ptr() + 2), dict(slots=q.data_ptr() + 1)):
            assert fi.lib.fi_lattn_prompt(op.handle, fi.fi_lattn_args(**{**ok, **kw})) == fi.FI_ERR_INVALID, kw
        assert fi.lib.fi_lattn_step(op.handle, fi.fi_lattn_args(**{**ok, "L": 1, "lens": q.data_ptr()})) == fi.FI_ERR_INVALID
        assert fi.lib.fi_lattn_prompt(op.handle, None) == fi.FI_ERR_INVALID
        assert fi.lib.fi_lattn_prompt(op.handle, fi.fi_lattn_args(**ok)) == fi.FI_OK
        torch.cuda.synchronize()


# ------------------------------------------------------------ dense product
def check_dense(seed, M, N, K, io="bf16", out="bf16", act="identity", bias=False, res=False, pad=0, shift=0, inplace=False):
    g, dt, ot = gen(seed), DT[io][0], DT[out][0]
    x = torch.randn(M, K, generator=g).to(dt)
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(dt)
    b = torch.randn(N, generator=g).to(dt) if bias else None
    r = torch.randn(M, N, generator=g).to(ot) if res else None
    ry, err = ref.dense(x, w, b, act, r)

    def dev(a, p=pad):
        buf = torch.full((a.shape[0], a.shape[1] + p + shift), float("nan"), dtype=a.dtype, device="cuda")
        v = buf[:, shift:shift + a.shape[1]]
        v.copy_(a)
        return v
    y = dev(torch.full((M, N), 3.0, dtype=ot)) if not inplace else dev(r)
    dres = y if inplace else dev(r) if res else None
    log("case dense", M, N, K, io, out, act, "bias", bias, "res", res, "pad", pad, "shift", shift)
    name = {"gelu": fi.FI_ACT_GELU, "tanh": fi.FI_ACT_TANH, "identity": fi.FI_ACT_IDENTITY}[act]
    with fi.Dense(M, N, K, DT[io][1], DT[out][1], name, stream()) as op:
        op.run(dev(x), dev(w), y, bias=None if b is None else b.cuda(), res=dres)
        torch.cuda.synchronize()
    got = y.cpu().double()
    u = ref.U16 if out == "bf16" else ref.U32
    over = ((got - ry).abs() - (err + u * (ry.abs() + err) + 1e-30)).max()
    log("dense max excess %.3g, rel l2 %.3g" % (over, ref.rel_l2(got, ry)))
    assert torch.isfinite(got).all() and float(over) <= 0.0
    if pad:
        base = y._base if y._base is not None else y
        assert bool(torch.isnan(base[:, shift + N:]).all())     # nothing beyond a row's end is written


@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 64), (1, 1000, 1024), (2, 129, 77), (3, 4096, 512), (8, 257, 1000),
                                   (16, 512, 2048), (17, 100, 96), (33, 640, 128), (65, 65, 65), (128, 256, 320),
                                   (300, 257, 130), (257, 1024, 64), (512, 512, 32), (1000, 48, 520)])
def test_dense_sizes(M, N, K, io, out):
    check_dense(M + N + K, M, N, K, io, out)


@pytest.mark.parametrize("act", ["gelu", "tanh", "identity"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 256), (5, 96, 100), (150, 200, 96), (256, 256, 256)])
@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_dense_epilogue(M, N, K, act, io, out):
    check_dense(M, M, N, K, io, out, act, bias=True, res=True)
    check_dense(M, M, N, K, io, out, act, bias=True)
    check_dense(M, M, N, K, io, out, act, res=True, inplace=True)


@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 8), (5, 1)])
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (9, 100, 90), (200, 300, 128), (256, 256, 136)])
def test_dense_strides(M, N, K, pad, shift, io, out):
    check_dense(M * pad, M, N, K, io, out, "gelu", bias=True, res=True, pad=pad, shift=shift)


@pytest.mark.parametrize("io,M,N,K", [
    ("bf16", 4090, 4050, 72), ("f32", 4090, 4050, 36), ("bf16", 2048, 4090, 200), ("f32", 2040, 2048, 100),      # tiles of 256, of 128
    ("bf16", 1024, 4090, 136), ("f32", 3606, 1071, 68), ("bf16", 2047, 4100, 75), ("f32", 2047, 2050, 37),       # 128 x 64; unaligned
    ("bf16", 64, 512, 4160), ("bf16", 200, 300, 3071), ("f32", 64, 260, 2100), ("f32", 40, 1000, 1027),          # parts of K
    ("bf16", 17, 9000, 264), ("bf16", 32, 500, 2056), ("f32", 25, 8200, 101), ("bf16", 16, 33000, 71)])          # few rows, either way
def test_dense_every_route(io, M, N, K):
    check_dense(M + K, M, N, K, io, io, "gelu", bias=True, res=True)


def test_dense_fewer_rows_than_the_config():
    x, w = torch.randn(4, 32, device="cuda"), torch.randn(16, 32, device="cuda")
    y = torch.full((4, 16), 9.0, device="cuda")
    with fi.Dense(4, 16, 32, fi.FI_F32, fi.FI_F32, stream=stream()) as op:
        op.run(x[:0], w, y[:0])
        op.run(x[:3], w, y[:3])
        torch.cuda.synchronize()
    assert bool((y[3] == 9.0).all())
    assert ref.rel_l2(y[:3], x[:3].cpu().double() @ w.cpu().double().t()) <= 1e-6


def test_dense_refusals():
    x, w, y = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda"), torch.zeros(4, 6, device="cuda")
    with fi.Dense(4, 6, 8, fi.FI_F32, fi.FI_F32, stream=stream()) as op:
        ok = dict(M=4, x=x.data_ptr(), ldx=8, w=w.data_ptr(), ldw=8, y=y.data_ptr(), ldy=6)
        for kw in (dict(M=5), dict(M=-1), dict(x=0), dict(w=0), dict(y=0), dict(ldx=7), dict(ldw=7), dict(ldy=5),
                   dict(res=y.data_ptr(), ldr=5), dict(x=x.data_ptr() + 2), dict(y=y.data_ptr() + 1),
                   dict(bias=x.data_ptr() + 2), dict(ldx=1 << 60)):
            assert fi.lib.fi_dense_run(op.handle, fi.fi_dense_args(**{**ok, **kw})) == fi.FI_ERR_INVALID, kw
        assert fi.lib.fi_dense_run(op.handle, None) == fi.FI_ERR_INVALID
        for a in ((x, w[:5], y), (x, w, y[:3]), (x[:, :7], w, y), (x, w, y[:, :5]), (x.t().contiguous().t(), w, y)):
            with pytest.raises(fi.FiError) as e:
                op.run(*a)
            assert e.value.status == fi.FI_ERR_INVALID
        assert fi.lib.fi_dense_run(op.handle, fi.fi_dense_args(**ok)) == fi.FI_OK
        torch.cuda.synchronize()


# ------------------------------------------------------------ token scores
def check_scores(logits, targets, k, dtype, scale=1.0, pad=0, shift=0):
    R, V = logits.shape
    dt = DT[dtype][0]
    logits = logits.to(dt)
    buf = torch.full((R, V + pad + shift), float("nan"), dtype=dt, device="cuda")
    buf[:, shift:shift + V] = logits.cuda()
    z = buf[:, shift:shift + V]
    lp, H, lse = (torch.full((R,), 9.0, device="cuda") for _ in range(3))
    top = torch.full((R, k), 9.0, device="cuda") if k else None
    ids = torch.full((R, k), 9, dtype=torch.int64, device="cuda") if k else None
    log("case scores", R, V, "k", k, dtype, "scale", scale, "pad", pad, "shift", shift)
    with fi.TokenScores(R, V, k, DT[dtype][1], scale, stream()) as op:
        op.run(z, targets.cuda(), lp, H, top, ids, lse)
        torch.cuda.synchronize()
    rlp, rH, rlse, rtop, rids = ref.scores(logits, targets, k, torch.tensor(scale).item())

    def near(got, want, a, b, what):
        got, want = got.cpu().double(), want
        assert torch.equal(torch.isnan(got), torch.isnan(want)), what
        f = torch.isfinite(want.float())   # a value beyond fp32's range is infinite in an fp32 output
        want = torch.where(f, want, want.float().double())
        assert torch.equal(got[~f & ~torch.isnan(want)], want[~f & ~torch.isnan(want)]), what
        assert bool(((got - want).abs()[f] <= a + b * want.abs()[f]).all()), (what, float((got - want).abs()[f].max()))
    near(lp, rlp, 8e-6, 1e-6, "logprob")
    near(H, rH, 4e-6, 1e-6, "entropy")
    near(lse, rlse, 4e-6, 1e-6, "lse")
    if k:
        assert torch.equal(ids.cpu(), rids)
        near(top, rtop, 8e-6, 1e-6, "top")


def logits_of(seed, R, V, spread=3.0):
    g = gen(seed)
    return torch.randn(R, V, generator=g) * spread, torch.randint(0, V, (R,), generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (3, 2, 5), (5, 7, 7), (2, 64, 32), (4, 255, 20), (3, 1000, 1), (7, 1025, 8),
                                   (1, 32001, 32), (300, 515, 4), (2, 131075, 20), (1, 262147, 5), (40, 9000, 0)])
def test_scores_sizes(R, V, k, dtype):
    z, t = logits_of(V, R, V)
    check_scores(z, t, k, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(5, 0), (8, 0), (3, 1), (16, 8)])
def test_scores_strides(pad, shift, dtype):
    z, t = logits_of(pad, 5, 3001)
    check_scores(z, t, 6, dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 4096, 50001])
def test_scores_ties_go_to_the_lowest_index(V, dtype):
    g = gen(V)
    check_scores(torch.randint(-3, 3, (4, V), generator=g).float(), torch.randint(0, V, (4,), generator=g), 32, dtype)
    check_scores(torch.zeros(2, V), torch.tensor([0, V - 1]), 32, dtype)
    up = torch.arange(V).float().repeat(2, 1) / V * 8      # every later token is better
    check_scores(torch.cat([up, -up]), torch.tensor([0, 1, 2, V - 1]), 20, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_masks(dtype):
    """Tokens ruled out by -inf or by the type's lowest value: all of a row,
    all but one, all but fewer than k; and a target that is ruled out."""
    V, k = 5000, 8
    z, t = logits_of(20, 8, V)
    z[0] = -math.inf
    z[1] = -math.inf
    z[1, 4321] = -5.0
    z[2, torch.arange(V) % 1000 != 7] = -math.inf
    z[3, :4999] = torch.finfo(DT[dtype][0]).min
    z[4] = torch.finfo(DT[dtype][0]).min
    z[5, 100:] = -math.inf
    t[1], t[5], t[6], t[7] = 4321, 2000, -1, -100
    check_scores(z, t, k, dtype)
    check_scores(z[:, :40], t.clamp(max=39), 20, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_not_finite(dtype):
    V = 3000
    z, t = logits_of(21, 6, V)
    z[0, 17] = float("nan")
    z[1, 2999] = math.inf
    z[2, 5], z[2, 6] = math.inf, float("nan")
    z[3] = float("nan")
    t[3], t[4], t[5] = -1, V, V + 7
    check_scores(z, t, 5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.5, 1.7, 8.0, 1e-3])
def test_scores_temperature(scale, dtype):
    z, t = logits_of(22, 4, 2500)
    check_scores(z, t, 9, dtype, scale=scale)


def test_scores_large_logits():
    z, t = logits_of(23, 4, 2500, spread=1.0)
    check_scores(z * 0.25 + 1.0e4, t, 9, "f32")
    check_scores(z * 40.0 - 3.0e4, t, 9, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("B,L,H,Hkv,dk,dv", [(2, 40, 320, 64, 8, 24), (3, 600, 14, 2, 24, 40), (2, 300, 15, 3, 96, 40), (1, 530, 7, 1, 200, 140)])
def test_prompt_shared_heads(B, L, H, Hkv, dk, dv, fresh, dtype):
    """Groups whose query heads go to several workgroups, also in shares that
    are not equal; rows that end early or hold nothing."""
    check_lattn(lattn_inputs(61, B, L, H, Hkv, dk, dv, dtype), dtype, lens=[L // 3, 0, L][:B], fresh=fresh)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fresh", [True, False])
def test_prompt_of_one_position(fresh, dtype):
    """Rows with one position, with none and without a state of the array."""
    inputs = lattn_inputs(63, 4, 1, 6, 2, 70, 33, dtype, slots=5)
    check_lattn(inputs, dtype, lens=[1, 0, 3, 1], slots=[4, 0, 2, 9], fresh=fresh)
    q, k, v, ld, state = inputs
    q[1], k[1], v[1] = float("nan"), float("nan"), float("inf")    # past the end of a row: not read as numbers
    check_lattn((q, k, v, ld, state), dtype, lens=[1, 0, 3, 1], slots=[4, 0, 2, 9], fresh=fresh)


@pytest.mark.parametrize("dtype,L", [("bf16", 2049), ("bf16", 2600), ("f32", 1025), ("f32", 4200)])
@pytest.mark.parametrize("dk,dv,fresh", [(40, 72, True), (136, 24, False)])
def test_prompt_many_segments(dtype, L, dk, dv, fresh):
    """Rows of so many chunks that a segment has several, and the last fewer."""
    check_lattn(lattn_inputs(62, 2, L, 2, 1, dk, dv, dtype), dtype, lens=[L - 70, L], fresh=fresh)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 40000])
@pytest.mark.parametrize("size, scale", [(1.0e7, 1.0), (2.0e7, 1.0), (1.0e10, 1.0), (1.0e17, 1.0), (1.0e29, 1.0), (1.0e38, 1.0),
                                         (100.0, 1.0e8), (1.0e-3, 1.0e20)])
def test_scores_huge_logits(V, size, scale, dtype):
    """Scaled logits beyond the whole numbers of fp32, up to its largest, of
    either sign, with the largest three times in two of the rows; in the last
    row only the part of the largest is huge."""
    g = torch.Generator().manual_seed(77)
    z = torch.randn(5, V, generator=g).clamp(-3.0, 3.0) * size
    z[1] = -z[1].abs() - size / 8
    for r in (0, 1):
        z[r, [V // 3, V // 2, V - 2]] = z[r].max()
    z[4] = torch.randn(V, generator=g) / scale
    z[4, 2 * V // 3] = size
    t = torch.randint(0, V, (5,), generator=g)
    t[0], t[4] = V // 2, 2 * V // 3
    check_scores(z, t, 6, dtype, scale=scale)


def test_scores_left_out_outputs():
    z, t = logits_of(24, 3, 400)
    zd, td = z.cuda(), t.cuda()
    H = torch.empty(3, device="cuda")
    rlp, rH, rlse, rtop, rids = ref.scores(z, t, 4)
    with fi.TokenScores(3, 400, 0, fi.FI_F32, stream=stream()) as op:
        op.run(zd, entropy=H)
        torch.cuda.synchronize()
        assert ref.rel_l2(H, rH) <= 1e-5
        lp = torch.empty(3, device="cuda")
        op.run(zd, td, lp)
        op.run(zd[:0], td[:0], lp[:0])
        torch.cuda.synchronize()
        assert ref.rel_l2(lp, rlp) <= 1e-5
        a = dict(rows=3, logits=zd.data_ptr(), ld=400)
        for kw in (dict(rows=4), dict(rows=-1), dict(logits=0), dict(ld=399), dict(ld=1 << 60),
                   dict(targets=td.data_ptr()), dict(logprob=lp.data_ptr()), dict(logits=zd.data_ptr() + 2),
                   dict(targets=td.data_ptr() + 4, logprob=lp.data_ptr()), dict(entropy=H.data_ptr() + 1)):
            assert fi.lib.fi_scores_run(op.handle, fi.fi_scores_args(**{**a, **kw})) == fi.FI_ERR_INVALID, kw
        assert fi.lib.fi_scores_run(op.handle, None) == fi.FI_ERR_INVALID
        with pytest.raises(fi.FiError):
            op.run(zd[:, :399], entropy=H)
    with fi.TokenScores(3, 400, 4, fi.FI_F32, stream=stream()) as op:
        with pytest.raises(fi.FiError):
            op.run(zd, td, lp)                        # k > 0 without top and top_id
        top, ids = torch.empty(3, 4, device="cuda"), torch.empty(3, 4, dtype=torch.int64, device="cuda")
        op.run(zd, top=top, top_id=ids)
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu(), rids) and ref.rel_l2(top, rtop) <= 1e-5


# ------------------------------------------------------------ streams and graphs
def test_operators_in_a_graph_on_their_stream():
    """A step of a decoder (projection, mixer, head, scores) captured on a side
    stream and replayed: every replay equals the eager run bit for bit."""
    B, H, d, V = 3, 4, 32, 1000
    D = H * d
    g = gen(30)
    w = (torch.randn(3 * D, D, generator=g) / math.sqrt(D)).bfloat16().cuda()
    head = (torch.randn(V, D, generator=g) / math.sqrt(D)).bfloat16().cuda()
    x = torch.randn(B, D, generator=g).bfloat16().cuda()
    ld = torch.full((H,), -0.01, device="cuda")
    state0 = torch.randn(B, H, d, d, generator=g).cuda()
    state, qkv = state0.clone(), torch.empty(B, 3 * D, dtype=torch.bfloat16, device="cuda")
    o, logits = torch.empty(B, 1, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, V, device="cuda")
    ent, top, ids = torch.empty(B, device="cuda"), torch.empty(B, 4, device="cuda"), torch.empty(B, 4, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with fi.Dense(B, 3 * D, D, stream=side) as proj, fi.Dense(B, V, D, out_dtype=fi.FI_F32, stream=side) as lm, \
            fi.LinearAttention(B, 1, H, H, d, d, ld, 1.0, fi.FI_BF16, side) as mix, \
            fi.TokenScores(B, V, 4, fi.FI_F32, stream=side) as sc:
        def run():
            proj.run(x, w, qkv)
            q, k, v = (p.reshape(B, 1, H, d) for p in qkv.split(D, 1))
            mix.step(q, k, v, o, state)
            lm.run(o.reshape(B, D), head, logits)
            sc.run(logits, entropy=ent, top=top, top_id=ids)
        want = []
        with torch.cuda.stream(side):
            for _ in range(4):
                run()
                side.synchronize()
                want.append([t.clone() for t in (state, o, logits, ent, top, ids)])
            state.copy_(state0)
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                run()
            state.copy_(state0)
            for i in range(4):
                graph.replay()
                side.synchronize()
                for a, b in zip((state, o, logits, ent, top, ids), want[i]):
                    assert torch.equal(a, b), i
