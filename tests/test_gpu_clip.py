"""Gradient clipping by the global norm on the GPU, against plain definitions
in 64 bits on the same inputs.

Tolerances, from the number formats alone:
* norm: at most 64 squares (positive numbers) are added in binary32 before
  they join a binary64 sum, each addition within 2^-24 relative, so the sum is
  within 64 * 2^-24 = 2^-18, its root within 2^-19, and the one rounding to
  binary32 adds 2^-24;
* coef: the norm's tolerance and one division's 2^-24;
* everything else (clipped tensors, reduced gradients, the Adam state given
  the coef that the device computed) is one fixed sequence of binary32
  operations: bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import Guarded, bits32, f32, u16
from optimizer_state_gb300 import inputs as I

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -19 + 2.0 ** -24
COEF_TOL = NORM_TOL + 2.0 ** -24
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
B16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z3():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is not available: the GPU tests need a GPU")
    from optimizer_state_gb300 import build, z3
    build.build()
    z3.load()
    return z3


@pytest.fixture()
def clip():
    return torch.full((2,), -1.0, device="cuda")


@pytest.fixture(scope="module")
def ws(z3):
    """One workspace for all tests, full of NaN at first: nothing in it counts."""
    return z3.grad_norm_workspace().fill_(255)


def normal(n, std, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(n, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def exact_norm(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def check_norm(clip, want, max_norm):
    norm, coef = (float(x) for x in clip.cpu().double())
    assert abs(norm - want) <= NORM_TOL * want, (norm, want)
    if abs(want - max_norm) > 2 * NORM_TOL * want:
        exact = max_norm / want if want > max_norm else 1.0
        assert abs(coef - exact) <= COEF_TOL * exact, (coef, exact)
    # the definition on the device's own norm
    n32, m32 = np.float32(norm), np.float32(max_norm)
    assert np.float32(coef) == (m32 / n32 if n32 > m32 else np.float32(1))


def back_to_back(lengths, dtype, std, seed, shift=0):
    """Views of these lengths one after the other in one guarded buffer, the
    first `shift` elements past a 16-byte boundary."""
    buf = Guarded(shift + sum(lengths), dtype)
    buf.t.copy_(normal(buf.n, std, dtype, seed))
    views, at = [], shift
    for n in lengths:
        views.append(buf.t[at:at + n])
        at += n
    return buf, views


LISTS = [
    [1], [7], [8], [9], [35, 13, 12], [1] * 50, [0, 5, 0, 0, 3],
    [511, 512, 513, 4095, 4096, 4097],
    [16384 * 8 + 1],                       # one tensor over many CTAs
    [3, 1000003, 2, 65537, 1, 250007],
    [17] * 159, [17] * 160, [17] * 161,    # around the first launch table's size
    [5] * 1901,                            # more tensors than one launch takes
    [4099] * 200,
    # around what one CTA, eight of them and one cluster take, of either type
    [24576], [24577], [49151], [49152], [49153], [98304], [98305], [49100, 60, 49000, 200],
]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("lengths", LISTS, ids=lambda x: f"{len(x)}x{max(x)}")
def test_norm_and_clip(z3, clip, ws, lengths, dtype, shift):
    buf, views = back_to_back(lengths, dtype, 1e-3, seed=len(lengths) + shift, shift=shift)
    before = buf.t.clone()
    want = exact_norm([buf.t[shift:]])
    for max_norm in (0.37 * want, 2.0 * want):
        buf.t.copy_(before)
        tl = z3.TensorList(views)
        z3.z3_grad_norm(tl, max_norm, clip, ws)
        check_norm(clip, want, np.float32(max_norm))
        z3.z3_clip(tl, clip)
        scaled = (before.float() * clip[1]).to(dtype) if clip[1] != 1 else before
        scaled[:shift] = before[:shift]    # in front of the first tensor: not its own
        assert torch.equal(buf.t.view(torch.uint8), scaled.view(torch.uint8))
        assert buf.guards_intact()


def test_norm_of_mixed_types_gaps_and_orders(z3, clip, ws):
    """Tensors of both types, apart and in no order, some twice in the norm."""
    ts = [normal(n, 0.1, d, i) for i, (n, d) in enumerate(
        [(1001, F32), (77, B16), (70001, B16), (1, F32), (262147, F32), (5, B16)])]
    view = ts[2][333:40004]
    lst = [ts[4], ts[1], view, ts[0], ts[5], ts[3], ts[1]]
    want = exact_norm(lst)
    z3.z3_grad_norm(lst, 1.0, clip, ws)
    check_norm(clip, want, 1.0)
    with pytest.raises(z3.Z3Error, match="overlaps"):
        z3.z3_clip(lst, clip)
    keep = [t.clone() for t in ts]
    z3.z3_clip([ts[4], view, ts[0]], clip)
    assert torch.equal(ts[4], keep[4] * clip[1]) and torch.equal(ts[0], keep[0] * clip[1])
    assert torch.equal(view, (keep[2][333:40004].float() * clip[1]).to(B16))
    for i in (1, 3, 5):
        assert torch.equal(ts[i], keep[i])
    assert torch.equal(ts[2][:333], keep[2][:333]) and torch.equal(ts[2][40004:], keep[2][40004:])


def test_norm_of_nothing(z3, clip, ws):
    for lst in ([], [torch.empty(0, device="cuda")] * 3):
        clip.fill_(-1)
        z3.z3_grad_norm(lst, 1.0, clip, ws)
        assert clip.tolist() == [0.0, 1.0]
        z3.z3_clip(lst, clip)
    z = torch.zeros(100003, device="cuda")
    z3.z3_grad_norm([z], 1.0, clip, ws)
    assert clip.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("std", [1e30, 3e36, 1e-20, 1e-30, 1e-38, 3e-40])
def test_norm_beyond_the_range_of_binary32_squares(z3, clip, ws, dtype, std):
    """Values whose squares overflow or vanish in binary32, down to subnormals."""
    for n in (5, 100003):
        t = normal(n, std, F32, 1).to(dtype)
        want = exact_norm([t])
        if want > 3e38:
            continue
        max_norm = 0.25 * want
        if max_norm < 1e-37:                # a normal binary32 number
            max_norm = 1e-37
        z3.z3_grad_norm([t], max_norm, clip, ws)
        norm = float(clip[0].double())
        spacing = 2.0 ** -149               # of subnormal binary32 norms
        assert abs(norm - want) <= NORM_TOL * want + spacing
        # mixed with ordinary values, and the two extremes together
        both = [t, normal(777, 1.0, dtype, 2), normal(3, 1e-35, dtype, 3)]
        want = exact_norm(both)
        z3.z3_grad_norm(both, 1.0, clip, ws)
        assert abs(float(clip[0].double()) - want) <= NORM_TOL * want


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 4242, 99999])
def test_a_norm_that_is_not_finite_stops_the_step(z3, clip, ws, dtype, bad, at):
    t = normal(100000, 1.0, dtype, 3)
    t[at] = bad
    keep = t.clone()
    z3.z3_grad_norm([t], 1.0, clip, ws)
    norm, coef = clip.tolist()
    assert math.isnan(coef)
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    z3.z3_clip([t], clip)
    assert torch.equal(t.view(torch.uint8), keep.view(torch.uint8))
    # nothing of it stays for the next call
    t[at] = 0
    z3.z3_grad_norm([t], 1.0, clip, ws)
    check_norm(clip, exact_norm([t]), 1.0)


def test_a_norm_beyond_binary32_counts_as_not_finite(z3, clip, ws):
    t = torch.full((1000,), 3e38, device="cuda")
    z3.z3_grad_norm([t], 1.0, clip, ws)
    assert clip[0] == math.inf and clip[1].isnan()


def test_infinite_max_norm_only_measures(z3, clip, ws):
    t = normal(5000, 1.0, F32, 4)
    z3.z3_grad_norm([t], math.inf, clip, ws)
    assert clip[1] == 1.0
    check_norm(clip, exact_norm([t]), math.inf)


def test_same_call_same_bits_and_stream_and_graph(z3, clip, ws):
    _, views = back_to_back([70001, 3, 250007, 5, 1000003], F32, 1e-3, 5, shift=1)
    tl = z3.TensorList(views)
    z3.z3_grad_norm(tl, 0.01, clip, ws)
    first = clip.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros(64, 4, device="cuda")
    for i in range(32):
        z3.z3_grad_norm(tl, 0.01, out[i, :2], ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(32, 64):
            z3.z3_grad_norm(tl, 0.01, out[i, :2], ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:, :2], first.expand(64, 2)) and not out[:, 2:].any()


@pytest.mark.parametrize("lengths", [[7], [5000, 3], [17] * 300, [100003, 65537]])
def test_norm_and_clip_in_turn(z3, clip, ws, lengths):
    """Forty times one after the other without a wait: every norm is of what
    the clipping before it wrote."""
    _, views = back_to_back(lengths, F32, 1.0, 8, shift=1)
    tl = z3.TensorList(views)
    out = torch.zeros(40, 4, device="cuda")
    want = [exact_norm(views) * 0.9 ** (i + 1) for i in range(40)]
    for i in range(40):
        z3.z3_grad_norm(tl, want[i], out[i, :2], ws)
        z3.z3_clip(tl, out[i, :2])
    got = out[1:, 0].cpu().double().numpy()
    # each pass rounds every element once more, by 2^-24 at most, and coef too
    assert np.all(np.abs(got / want[:-1] - 1) <= NORM_TOL + COEF_TOL + 2.0 ** -23)


def test_nan_in_an_earlier_launch_of_a_long_list(z3, clip, ws):
    _, views = back_to_back([5] * 4000, B16, 1.0, 9)
    z3.z3_grad_norm(views, 1.0, clip, ws)
    check_norm(clip, exact_norm(views), 1.0)
    views[3][2] = math.nan
    z3.z3_grad_norm(views, 1.0, clip, ws)
    assert clip.isnan().all()


def test_a_tensor_longer_than_32_bits(z3, clip, ws):
    n = 2 ** 32 + 11                        # 8.6 GB of bf16
    t = torch.zeros(n, dtype=B16, device="cuda")
    places = [0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 1]
    for i, x in enumerate(places):
        t[x] = 2.0 ** i
    z3.z3_grad_norm([t], 1.0, clip, ws)
    check_norm(clip, math.sqrt(sum(4.0 ** i for i in range(len(places)))), 1.0)
    z3.z3_clip([t], clip)
    for i, x in enumerate(places):
        assert t[x] == torch.tensor(2.0 ** i * float(clip[1]), dtype=B16)
    assert int(t.count_nonzero()) == len(places)


# ---------------------------------------------------------------------------
# the reduce-scatter with its sums of squares
# ---------------------------------------------------------------------------

LAYERS = [([35, 13, 12], 4), ([1], 64), ([1, 1, 2], 3), ([4096, 8192, 64], 8), ([262147], 2),
          ([100003, 7, 4099], 3), ([0, 5, 0, 70001], 16), ([50257, 1024], 1),
          ([64] * 40 + [7, 56], 8), ([8192 + 3] * 45, 64)]


def layer_grads(w, seed):
    return I.draw_grads(w, I.make_generator(seed, "cuda"), "cuda")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("numel,ranks", LAYERS, ids=lambda x: str(x)[:24])
def test_reduce_scatter_norm(z3, orc, clip, ws, numel, ranks, accumulate):
    w = I.Workload("case", tuple((n,) for n in numel), ranks, 0.02, 1e-3)
    L, O = z3.Layout(numel, ranks), orc.layout(numel, ranks)
    grads = layer_grads(w, 3)
    out = Guarded(L.psi_padded, F32)
    sq = torch.full((L.sumsq_len + 2,), math.nan, dtype=torch.float64, device="cuda")
    out.t.zero_()
    host = np.zeros(L.psi_padded, np.float32)
    if accumulate:
        first = layer_grads(w, 4)
        z3.z3_reduce_scatter(L, first, w.grad_stride, out.t, 0.5)
        host = orc.reduce_scatter(O, u16(first).reshape(-1), w.grad_stride, 0.5)
    else:
        out.t.fill_(math.nan)               # what was there is not read
    z3.z3_reduce_scatter_norm(L, grads, w.grad_stride, out.t, 0.5, sq[:L.sumsq_len],
                              accumulate=accumulate)
    host = orc.reduce_scatter(O, u16(grads).reshape(-1), w.grad_stride, 0.5, out=host,
                              accumulate=accumulate)
    assert np.array_equal(bits32(f32(out.t)), bits32(host))
    assert out.guards_intact() and sq[L.sumsq_len:].isnan().all()
    want = math.sqrt(float(np.square(host.astype(np.float64)).sum()))
    got = math.sqrt(float(sq[:L.sumsq_len].sum()))
    assert abs(got - want) <= NORM_TOL * want
    extra = normal(333, 1e-3, B16, 9)       # gradients from elsewhere join the norm
    z3.z3_grad_norm(z3.TensorList([extra], sumsq=[sq[:L.sumsq_len]]), 1e-3, clip, ws)
    check_norm(clip, math.hypot(want, exact_norm([extra])), 1e-3)


@pytest.mark.parametrize("std", [1e25, 1e-30])
def test_reduce_scatter_norm_beyond_binary32_squares(z3, clip, ws, std):
    w = I.Workload("case", ((70001,), (11,)), 4, 0.02, std)
    L = z3.Layout(w.numel, 4)
    grads, out = layer_grads(w, 5), torch.empty(L.psi_padded, device="cuda")
    sq = torch.empty(L.sumsq_len, dtype=torch.float64, device="cuda")
    z3.z3_reduce_scatter_norm(L, grads, w.grad_stride, out, 0.25, sq)
    want = exact_norm([out])
    z3.z3_grad_norm(z3.TensorList([], sumsq=[sq]), 1.0, clip, ws)
    check_norm(clip, want, 1.0)
    with pytest.raises(z3.Z3Error, match="sums of squares"):
        z3.z3_clip(z3.TensorList([], sumsq=[sq]), clip)
    for bad in (math.inf, math.nan):
        grads[2, 70003] = bad
        z3.z3_reduce_scatter_norm(L, grads, w.grad_stride, out, 0.25, sq)
        z3.z3_grad_norm(z3.TensorList([], sumsq=[sq]), 1.0, clip, ws)
        assert clip[1].isnan() and not clip[0].isfinite()


# ---------------------------------------------------------------------------
# the clipped update
# ---------------------------------------------------------------------------

def draw_state(L, seed):
    T = L.psi_padded
    st = dict(master=Guarded(T, F32), m=Guarded(T, F32), v=Guarded(T, F32), shards=Guarded(T, B16))
    st["master"].t.copy_(normal(T, 0.02, F32, seed))
    st["m"].t.copy_(normal(T, 1e-3, F32, seed + 1))
    st["v"].t.copy_(normal(T, 1e-3, F32, seed + 2).square())
    st["shards"].t.copy_(st["master"].t)
    return st


def host_state(st):
    return {k: (u16 if k == "shards" else f32)(b.t).copy() for k, b in st.items()}


def oracle_adam(orc, h, g, t):
    orc.adam(h["master"], h["m"], h["v"], g, h["shards"], HP["lr"], HP["beta1"], HP["beta2"],
             HP["eps"], HP["weight_decay"], t)


def assert_state(st, want):
    got = host_state(st)
    for k in want:
        bits = np.uint16 if k == "shards" else np.uint32
        assert np.array_equal(got[k].view(bits), want[k].view(bits)), k
        assert st[k].guards_intact(), k


@pytest.mark.parametrize("coef", [1.0, 0.43, 1e-20, 0.0, math.nan])
@pytest.mark.parametrize("numel,ranks", [([35, 13, 12], 4), ([1], 1), ([262147], 2),
                                         ([100003, 7], 3)])
def test_adam_clipped(z3, orc, numel, ranks, coef):
    L = z3.Layout(numel, ranks)
    st = draw_state(L, 11)
    want = host_state(st)
    g = normal(L.psi_padded, 1e-3, F32, 7)
    keep = g.clone()
    clip = torch.tensor([5.0, coef], device="cuda")
    z3.z3_adam_shard_step_clipped(L, st["master"].t, st["m"].t, st["v"].t, g, st["shards"].t, HP,
                                  4, clip)
    if not math.isnan(coef):
        oracle_adam(orc, want, f32(g) * np.float32(coef), 4)
    assert_state(st, want)
    assert torch.equal(g, keep)


# ---------------------------------------------------------------------------
# the whole clipped step
# ---------------------------------------------------------------------------

UNITS = [((4096,), (64,)), ((100003,), (7,), (4099,)), ((0,),), ((8192 + 3,),), ((1,),)]


def make_model(prefetch, resident=(), seed=1, ranks=4):
    from optimizer_state_gb300 import schedule
    gen = I.make_generator(seed, "cuda")
    units = [schedule.Unit(I.Workload(f"u{i}", s, ranks, 0.02, 1e-3, resident=i in resident),
                           torch.device("cuda"), gen) for i, s in enumerate(UNITS)]
    dev = torch.device("cuda")
    return schedule.PrefetchModel(units, dev, prefetch) if prefetch else schedule.Model(units, dev)


def model_bits(m):
    torch.cuda.synchronize()
    return [(u16(u.shards), bits32(f32(u.master)), bits32(f32(u.m)), bits32(f32(u.v)),
             None if u.resident is None else u16(u.resident)) for u in m.units]


def same(a, b):
    return all(np.array_equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q) if x is not None)


@pytest.mark.parametrize("prefetch,resident", [(0, ()), (0, (3,)), (1, ()), (2, (0, 4))])
def test_clipped_model_step(z3, orc, prefetch, resident):
    """Three steps against the oracle: reduce, the norm of every unit in 64
    bits, then Adam with the device's own coef; one is not clipped."""
    m = make_model(prefetch, resident)
    host = []
    for u in m.units:
        host.append(dict(O=orc.layout(u.L.numel, u.L.n_ranks), shards=u16(u.shards).copy(),
                         master=f32(u.master).copy(), m=f32(u.m).copy(), v=f32(u.v).copy()))
    for t, max_norm in ((1, 0.05), (2, 1e3), (3, 1e-4)):
        m.step(HP, max_norm=max_norm)
        torch.cuda.synchronize()
        reduced = [orc.reduce_scatter(h["O"], u16(u.grads).reshape(-1), u.w.grad_stride,
                                      1.0 / u.w.n_ranks) for h, u in zip(host, m.units)]
        want = math.sqrt(sum(float(np.square(g.astype(np.float64)).sum()) for g in reduced))
        check_norm(m.clip, want, np.float32(max_norm))
        coef = np.float32(float(m.clip[1]))
        for h, u, g in zip(host, m.units, reduced):
            oracle_adam(orc, h, g * coef, t)
            assert np.array_equal(u16(u.shards), h["shards"])
            for k in ("master", "m", "v"):
                assert np.array_equal(bits32(f32(getattr(u, k))), bits32(h[k])), k
            if u.resident is not None:
                assert np.array_equal(u16(u.resident), orc.allgather(h["O"], h["shards"]))


@pytest.mark.parametrize("prefetch", [0, 2])
def test_unclipped_and_stopped_steps(z3, prefetch):
    """A bound that is not reached gives z3_model_step's state bit for bit; a
    gradient that is not finite leaves the state as it was."""
    a, b = make_model(prefetch, (1,)), make_model(prefetch, (1,))
    a.step(HP)
    b.step(HP, max_norm=1e6)
    assert same(model_bits(a), model_bits(b)) and b.clip[1] == 1.0
    before = model_bits(b)
    b.units[1].grads[2, 100005] = math.inf
    b.step(HP, max_norm=1e6)
    assert same(before, model_bits(b))
    assert b.clip[0] == math.inf and b.clip[1].isnan()


@pytest.mark.parametrize("prefetch", [0, 1])
@pytest.mark.parametrize("max_norm", [0.01, 1e6])
def test_clipped_step_issued_call_by_call(z3, prefetch, max_norm):
    """The schedule with hooks, from Python, gives the library's step."""
    a, b = make_model(prefetch, (1,)), make_model(prefetch, (1,))
    seen = []
    for _ in range(2):
        a.step(HP, max_norm=max_norm)
        b.step(HP, max_norm=max_norm, on_gather=lambda phase, i: seen.append((phase, i)))
    assert same(model_bits(a), model_bits(b)) and torch.equal(a.clip, b.clip)
    n = len(UNITS)
    assert sorted(seen) == sorted(2 * [(p, i) for p in ("backward", "forward") for i in range(n)])


def test_clipped_step_of_many_units(z3):
    """More units than one launch's tables of the norm and of the update hold."""
    from optimizer_state_gb300 import schedule
    dev = torch.device("cuda")

    def model():
        gen = I.make_generator(2, "cuda")
        return schedule.Model([schedule.Unit(I.Workload(f"u{i}", ((i % 7 * 11,), (300,)), 3, 0.02,
                                                        1e-3), dev, gen) for i in range(190)], dev)
    a, b, c = model(), model(), model()
    a.step(HP)
    b.step(HP, max_norm=1e6)
    assert same(model_bits(a), model_bits(b))
    want = exact_norm([gs for gs, _ in b.clip_args()])
    check_norm(b.clip, want, 1e6)
    c.step(HP, max_norm=0.5 * want)
    check_norm(c.clip, want, np.float32(0.5 * want))
    c2 = model()
    c2.step(HP, max_norm=0.5 * want, on_gather=lambda *a: None)
    assert same(model_bits(c), model_bits(c2)) and not same(model_bits(b), model_bits(c))


def test_clipped_step_of_empty_units(z3, clip, ws):
    L = z3.Layout([0], 4)
    e = torch.empty(0, device="cuda")
    unit = (L, e.to(B16), e, e, e, e.to(B16), 0, 0.25)
    sq = torch.empty(0, dtype=torch.float64, device="cuda")
    z3.z3_model_step_clipped([unit, unit], [(e, sq)] * 2, [torch.empty(8, dtype=B16, device="cuda")],
                             HP, 1, 1.0, clip, ws)
    assert clip.tolist() == [0.0, 1.0]


def test_clipped_step_accumulates_micro_batches(z3, orc, clip, ws):
    """Micro-batches before the last go through z3_reduce_scatter; the last
    one's clipped step adds to them."""
    m = make_model(0)
    args = m.clip_args()
    sums = []
    for u, (gs, _) in zip(m.units, args):
        z3.z3_reduce_scatter(u.L, u.grads, u.w.grad_stride, gs, 0.125)
        sums.append(f32(gs).copy())
        u.grads.mul_(0.5)
    z3.z3_model_step_clipped(m.unit_args(), [(*c, True) for c in args], [m.full], HP, 1, 0.01,
                             clip, ws)
    for u, (gs, _), s in zip(m.units, args, sums):
        O = orc.layout(u.L.numel, u.L.n_ranks)
        s = orc.reduce_scatter(O, u16(u.grads).reshape(-1), u.w.grad_stride, 0.25, out=s,
                               accumulate=True)
        assert np.array_equal(bits32(f32(gs)), bits32(s))
    check_norm(clip, exact_norm([gs for gs, _ in args]), 0.01)


def test_clipped_step_in_a_graph(z3):
    a, b = make_model(0), make_model(0)
    a.clip_args(), b.clip_args()
    for t in (1, 2, 3):
        a.step(HP, t=t, max_norm=0.01)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t in (1, 2, 3):
            b.step(HP, t=t, max_norm=0.01)
    g.replay()
    assert same(model_bits(a), model_bits(b)) and torch.equal(a.clip, b.clip)
