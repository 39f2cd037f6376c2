"""Prompts of the gated delta rule that are split into segments (16 chunks and more of few heads), at head sizes that no kernel
is as wide as, unaligned views, rows that end in other segments, and several runs of chunks; held single tokens.
Against the recurrence in 64 bits, with the bounds of tests/test_gpu_delta.py: what a segment does to the state
before it is a product of terms that do not grow, and is added up as the state itself is."""
import pytest

import draft_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402  (fails loudly if libfi.so is missing)
from fi_harness import log  # noqa: E402
from op_reference import rel_l2  # noqa: E402
from test_gpu_delta import DT, TOL_STATE, check, check_output, inputs, stream  # noqa: E402

HEADS = [(1, 1), (33, 7), (80, 48), (64, 100), (64, 256), (100, 128), (128, 72), (130, 250), (192, 40), (192, 192), (256, 256)]


@pytest.mark.parametrize("dtype,L", [("bf16", 1300), ("f32", 700)])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_heads(dk, dv, fresh, dtype, L):
    check(inputs(dk + dv, 1, L, 1, 2, dk, dv, dtype, memory=(50.0, 3000.0)), dtype, fresh=fresh)


@pytest.mark.parametrize("dtype,L", [("bf16", 2500), ("f32", 1300)])
@pytest.mark.parametrize("dk,dv", [(33, 7), (100, 128), (256, 256)])
def test_more_segments(dk, dv, dtype, L):
    x = inputs(dk * dv, 2, L, 2, 2, dk, dv, dtype, memory=(500.0, 1e5))
    check(x, dtype, lens=[L, L - 700])
    check(x, dtype, hold=True)


@pytest.mark.parametrize("dtype,L", [("bf16", 1300), ("f32", 700)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 128)])
def test_misaligned_views(dk, dv, dtype, L):
    """Head sizes of whole 16-byte units, at an odd place in odd rows."""
    x = inputs(dk, 1, L, 2, 2, dk, dv, dtype)
    whole = torch.cat([y.reshape(1, L, -1) for y in x[:3]], -1)
    buf = torch.full((1, L, whole.shape[-1] + 3), float("nan"), dtype=whole.dtype, device="cuda")
    buf[..., 1:-2] = whole.cuda()
    parts = buf[..., 1:-2].split([2 * dk, 2 * dk, 2 * dv], -1)
    check(x, dtype, dev=tuple(p.unflatten(-1, (2, d)) for p, d in zip(parts, (dk, dk, dv))) + (x[3].cuda(), x[4].cuda()))


@pytest.mark.parametrize("dtype,L", [("bf16", 1300), ("f32", 700)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (48, 130), (256, 64)])
def test_ragged_rows_and_slots(dk, dv, dtype, L):
    """Rows without positions, that end in the first segment, at a segment's end, one before the last, out of the pool; NaN past their ends."""
    lens, slots = [L, 0, 1, L // 3, -3, L - 1, 256, 5000], [8, 0, 5, 3, 2, 7, 4, -1]
    x = inputs(3, 8, L, 1, 2, dk, dv, dtype, slots=9)
    dev = []
    for y in x[:5]:
        y = y.clone()
        for b in range(8):
            y[b, max(0, min(L, lens[b])):] = float("nan")
        dev.append(y.cuda())
    check(x, dtype, lens=lens, slots=slots, dev=dev)
    check(x, dtype, lens=lens, slots=slots, dev=dev, hold=True)
    slots[-1] = 6
    o, st = check(x, dtype, lens=lens, slots=slots, dev=dev, fresh=True)
    assert float(st[0].abs().max()) == 0.0 and float(st[2].abs().max()) == 0.0 and float(o[1].abs().max()) == 0.0
    slots[-1] = 9
    check(x, dtype, lens=lens, slots=slots, dev=dev, fresh=True)


@pytest.mark.parametrize("dtype,L,ends", [("f32", 21400, 17000), ("bf16", 35300, 33000)])
@pytest.mark.parametrize("fresh,hold", [(False, False), (True, False), (False, True)])
def test_several_runs_in_segments(fresh, hold, dtype, L, ends):
    """64 heads in four segments, of which more chunks than are held at a time: the second run begins from what the
    first hands on, and has fewer chunks, some segments none."""
    check(inputs(20, 2, L, 4, 32, 16, 8, dtype, memory=(1000.0, 50000.0)), dtype, lens=[L, ends], fresh=fresh, hold=hold)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_that_hold(dtype):
    """A held step answers as one that moves and changes no state; rows may share one."""
    B, Hk, Hv, dk, dv = 4, 2, 4, 80, 48
    x = inputs(5, B, 1, Hk, Hv, dk, dv, dtype, slots=3)
    slots = [2, 0, 0, 3]
    ro, _ = ref.delta(*x[:5], torch.tensor(0.3).item(), x[5], slots=slots, hold=True)
    d, st = [y.cuda() for y in x[:5]], x[5].cuda()
    o = torch.full((B, 1, Hv, dv), 7.0, dtype=x[0].dtype, device="cuda")
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    log("case delta held step", dtype)
    with fi.DeltaRule(B, 1, Hk, Hv, dk, dv, 0.3, DT[dtype][1], stream()) as op:
        op.step(*d, o, st, slots=sl, hold=True)
        torch.cuda.synchronize()
        assert torch.equal(st.cpu(), x[5])
        check_output(o, ro, dtype, "o")
        o2 = torch.empty_like(o)
        op.step(*(y[:2] for y in d), o2[:2], st, slots=sl[:2])
        torch.cuda.synchronize()
    assert torch.equal(o[:2], o2[:2])
    _, rs = ref.delta(*(y[:2] for y in x[:5]), 0.3, x[5], slots=slots[:2])
    assert rel_l2(st[2], rs[2]) <= TOL_STATE and rel_l2(st[0], rs[0]) <= TOL_STATE and torch.equal(st[1].cpu(), x[5][1])
