"""Losses over a vocabulary on the GPU against 64-bit plain forms, within bounds
derived from the number formats (head_reference)."""
import itertools

import pytest
import torch

from head_reference import outside, reference
from optimizer_state_gb300 import z3

pytestmark = pytest.mark.gpu

GUARD = 64


class Guarded:
    """A [rows, cols] tensor whose rows lie `pitch` apart, inside a buffer of a
    canary value."""

    def __init__(self, rows, cols, dtype, pitch=None):
        self.pitch = pitch or cols
        self.rows, self.cols = rows, cols
        self.raw = torch.full((2 * GUARD + max(rows, 1) * self.pitch,), 77.0, dtype=dtype,
                              device="cuda")
        self.t = self.raw[GUARD:GUARD + rows * self.pitch].view(rows, self.pitch)[:, :cols]

    def intact(self):
        raw = self.raw.clone()
        raw[GUARD:GUARD + self.rows * self.pitch].view(self.rows, self.pitch)[:, :self.cols] = 77.0
        return bool((raw == 77.0).all())


def rows_apart(t, pitch):
    """The same matrix with its rows `pitch` apart; NaN between them."""
    out = torch.full((t.shape[0], pitch), float("nan"), dtype=t.dtype, device=t.device)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]


class Case:
    def __init__(self, n, v, d, k=0, seed=0, ignored=0.2, weighted=False, teacher=torch.float32,
                 index=torch.int64, tau=1.0, peak=6.0, apart=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.rand(*shape, device="cuda", generator=g)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, device="cuda", generator=g) * std
        self.n, self.v, self.d, self.k, self.tau = n, v, d, k, tau
        weight = normal(v, d, std=d ** -0.5).to(torch.bfloat16)
        words = (rand(n) * v).long().clamp(max=v - 1)
        hidden = (normal(n, d) + peak * rand(n, 1) * weight[words].float()).to(torch.bfloat16)
        out = rand(n) < ignored
        self.hidden = rows_apart(hidden, d + apart) if apart else hidden
        self.weight = rows_apart(weight, d + 2 * apart) if apart else weight
        self.weights = rand(n) + 0.25 if weighted else None
        self.targets = self.index = self.teacher = None
        if k:
            self.index = (rand(n, k) * v).long().clamp(max=v - 1)
            self.teacher = normal(n, k, std=2.0).to(teacher)
            self.index[rand(n, k) < 0.1] = -1
            self.index[out] = -100
            self.index = self.index.to(index)
        else:
            self.targets = words.masked_fill(out, -100).to(index)
        self.apart = apart

    def reference(self, **kw):
        return reference(self.hidden, self.weight, self.targets, self.index, self.teacher, self.tau,
                         self.weights, **kw)

    def outputs(self):
        f32 = torch.float32
        self.o = dict(loss=Guarded(1, self.n, f32), lse=Guarded(1, self.n, f32),
                      total=Guarded(1, 2, f32),
                      d_hidden=Guarded(self.n, self.d, torch.bfloat16, self.d + 3 * self.apart),
                      d_weight=Guarded(self.v, self.d, torch.bfloat16, self.d + self.apart))
        t = {x: y.t for x, y in self.o.items()}
        return t | {x: t[x][0] for x in ("loss", "lse", "total")}

    def forward(self, t, ws, stream=None):
        tail = dict(loss=t["loss"], lse=t["lse"], total=t["total"], workspace=ws,
                    weights=self.weights, stream=stream)
        if self.k:
            z3.z3_distill(self.hidden, self.weight, self.teacher, self.index, self.tau, **tail)
        else:
            z3.z3_xent(self.hidden, self.weight, self.targets, **tail)

    def grad(self, t, ws, scale=1.0, mean=True, stream=None):
        tail = dict(lse=t["lse"], total=t["total"] if mean else None, scale=scale,
                    d_hidden=t["d_hidden"], d_weight=t["d_weight"], workspace=ws,
                    weights=self.weights, stream=stream)
        if self.k:
            z3.z3_distill_grad(self.hidden, self.weight, self.teacher, self.index, self.tau, **tail)
        else:
            z3.z3_xent_grad(self.hidden, self.weight, self.targets, **tail)

    def workspace(self):
        """Filled with NaN: nothing of it is read before it is written."""
        ws = z3.head_workspace(self.n, self.d, self.v, k=self.k)
        ws.fill_(0xff)
        return ws

    def check(self, scale=1.0, mean=True):
        t, ws = self.outputs(), self.workspace()
        self.forward(t, ws)
        ws.fill_(0xff)
        self.grad(t, ws, scale, mean)
        torch.cuda.synchronize()
        assert outside(t, self.reference(scale=scale, mean=mean)) == {}
        assert all(x.intact() for x in self.o.values())
        return t


SIZES = [(1, 1, 8), (1, 2, 8), (3, 64, 64), (128, 256, 64), (127, 63, 72), (129, 257, 72),
         (1, 1000, 136), (2, 5003, 520), (300, 65, 200), (128, 1024, 512), (257, 1000, 64),
         (777, 5003, 136), (130, 300, 1032), (1500, 129, 8), (32, 777, 64), (33, 5003, 72),
         (100, 20011, 64), (16, 40009, 128), (300, 520, 520), (200, 300, 296), (150, 300, 1000),
         (600, 333, 1288), (140, 4000, 24), (2000, 5003, 1032), (1300, 20011, 520)]


@pytest.mark.parametrize("n,v,d", SIZES)
def test_xent(n, v, d):
    Case(n, v, d).check()


@pytest.mark.parametrize("n,v,d", SIZES)
def test_distill(n, v, d):
    Case(n, v, d, k=7, tau=2.0).check()


@pytest.mark.parametrize("k,teacher,index,tau,n,v", [
    (1, torch.float32, torch.int32, 1.0, 200, 3000), (2, torch.bfloat16, torch.int64, 4.0, 40, 700),
    (64, torch.bfloat16, torch.int32, 1.5, 300, 3000), (65, torch.float32, torch.int64, 0.5, 90, 999),
    (200, torch.float32, torch.int32, 2.0, 513, 4003), (1024, torch.bfloat16, torch.int64, 1.0, 33, 200),
    (1000, torch.float32, torch.int64, 3.0, 150, 20011)])
def test_lists(k, teacher, index, tau, n, v):
    """Lists of every length, longer than the vocabulary among them: words stand
    in them many times."""
    Case(n, v, 72, k=k, teacher=teacher, index=index, tau=tau, weighted=True).check(scale=0.3)


@pytest.mark.parametrize("n", [5, 100, 700])
@pytest.mark.parametrize("k", [0, 9])
def test_rows_apart_weights_and_index_types(n, k):
    for index, weighted, mean in itertools.product((torch.int32, torch.int64), (False, True),
                                                   (False, True)):
        Case(n, 1003, 136, k=k, tau=1.5 if k else 1.0, index=index, weighted=weighted, apart=8,
             seed=n).check(scale=-2.0, mean=mean)


@pytest.mark.parametrize("n", [7, 129, 600])
@pytest.mark.parametrize("k", [0, 5])
def test_rows_left_out_hold_anything(n, k):
    """NaN and infinities in the rows of tokens that are left out, and of those
    whose weight is 0, reach no gradient; all rows left out."""
    c = Case(n, 700, 72, k=k, ignored=0.5, weighted=True)
    out = (c.index < 0).all(dim=1) if k else c.targets < 0
    want = c.reference()
    c.hidden = c.hidden.clone()
    c.hidden[out] = float("nan")
    c.hidden[out.nonzero()[::2, 0]] = float("inf")
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    c.grad(t, ws)
    torch.cuda.synchronize()
    assert outside(t, want) == {}
    # a weight of 0: the loss stays, NaN where its row is
    zero = (~out).nonzero()[:3, 0]
    c.weights[zero] = 0.0
    want = c.reference()
    c.hidden[zero] = float("nan")
    c.forward(t, ws)
    c.grad(t, ws)
    torch.cuda.synchronize()
    assert bool(t["loss"][zero].isnan().all())
    t["loss"][zero] = want["loss"][0][zero].float()
    t["lse"][zero] = want["lse"][0][zero].float()
    assert outside(t, want) == {}
    # nothing counts
    if k:
        c.index.fill_(-1)
    else:
        c.targets.fill_(-1)
    c.hidden.fill_(float("nan"))
    c.forward(t, ws)
    c.grad(t, ws)
    torch.cuda.synchronize()
    assert all(bool((t[x] == 0).all()) for x in t)


def test_lists_of_extreme_logits():
    """The type's lowest value is a logit as any; -Inf leaves an entry out, and a
    list of nothing else its token; +Inf and NaN spoil theirs."""
    c = Case(40, 300, 64, k=6, ignored=0.0)
    low = torch.finfo(torch.float32).min
    c.index.clamp_(min=0)
    c.teacher[0] = low                              # a uniform list
    c.teacher[1, 1:] = low                          # one entry
    c.teacher[2, ::2] = -torch.inf
    c.teacher[3] = -torch.inf
    c.teacher[4] = torch.finfo(torch.float32).max
    c.teacher[5] = -torch.inf
    c.teacher[5, 3] = -1.0
    c.check()
    for row, bad in ((6, torch.inf), (7, float("nan"))):
        d = Case(40, 300, 64, k=6, ignored=0.0)
        d.teacher[row, 2] = bad
        d.index[row, 2] = 5
        t, ws = d.outputs(), d.workspace()
        d.forward(t, ws)
        d.grad(t, ws)
        torch.cuda.synchronize()
        assert bool(t["loss"][row].isnan()) and int(t["loss"].isnan().sum()) == 1
        assert bool(t["total"][0].isnan()) and bool(t["d_hidden"][row].isnan().all())


@pytest.mark.parametrize("n", [6, 300])
@pytest.mark.parametrize("k", [0, 4])
def test_words_beyond_the_vocabulary(n, k):
    """They read nothing, spoil their token's loss, and the weight's gradient."""
    for beyond in (301, 2 ** 31 - 1, 2 ** 40):
        c = Case(n, 301, 64, k=k, ignored=0.0)
        want = c.reference()["loss"]
        if k:
            c.index[2, 1] = beyond
        else:
            c.targets[2] = beyond
        t, ws = c.outputs(), c.workspace()
        c.forward(t, ws)
        c.grad(t, ws)
        torch.cuda.synchronize()
        assert bool(t["loss"][2].isnan()) and bool(t["total"][0].isnan())
        others = torch.arange(n, device="cuda") != 2
        assert bool(((t["loss"].double() - want[0]).abs() <= want[1])[others].all())
        assert bool(t["d_hidden"][2].isnan().all()) and bool(t["d_weight"].isnan().all())
        assert bool(t["d_hidden"][others].isfinite().all())
        assert all(x.intact() for x in c.o.values())


def test_logits_that_are_not_finite_spoil_their_token_alone():
    c = Case(200, 500, 64, ignored=0.0)
    want = c.reference()["loss"]
    c.hidden[3, 5] = float("inf")
    c.hidden[4, 5] = float("nan")
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    torch.cuda.synchronize()
    others = torch.ones(200, dtype=torch.bool, device="cuda")
    others[3:5] = False
    assert bool(t["loss"][3:5].isnan().all())
    assert bool(((t["loss"].double() - want[0]).abs() <= want[1])[others].all())


@pytest.mark.parametrize("k", [0, 3])
def test_no_tokens(k):
    c = Case(0, 50, 64, k=k)
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    c.grad(t, ws)
    torch.cuda.synchronize()
    assert t["total"].tolist() == [0.0, 0.0] and bool((t["d_weight"] == 0).all())
    assert all(x.intact() for x in c.o.values())


def test_several_pieces_of_the_vocabulary():
    """Sizes whose dz takes more than one piece, with a last one of odd length."""
    for n, v, d, k in ((6000, 50021, 24, 0), (9000, 30011, 40, 5)):
        assert n * v * 2 > 256 << 20
        Case(n, v, d, k=k).check()


@pytest.mark.parametrize("k", [0, 4])
def test_either_gradient_alone(k):
    c = Case(300, 900, 72, k=k)
    t = c.check()
    both = {x: t[x].clone() for x in ("d_hidden", "d_weight")}
    for x in both:
        t = c.outputs()
        ws = c.workspace()
        c.forward(t, ws)
        other = "d_weight" if x == "d_hidden" else "d_hidden"
        c.grad(t | {other: None}, ws)
        torch.cuda.synchronize()
        assert torch.equal(t[x], both[x])
        assert bool((t[other] == 77.0).all())


@pytest.mark.parametrize("n,k", [(20, 0), (20, 6), (900, 0), (900, 6)])
def test_the_same_bits_on_any_stream_and_replayed(n, k):
    """Eager on two streams at a time, each with its workspace, and captured and
    replayed on other inputs: the same bits."""
    c = Case(n, 4001, 136, k=k)
    first = {x: y.clone() for x, y in c.check().items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    runs = [(c.outputs(), c.workspace()) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (t, ws) in zip(streams, runs):
            c.forward(t, ws, stream=s)
            c.grad(t, ws, stream=s)
    torch.cuda.synchronize()
    for t, _ in runs:
        assert all(torch.equal(t[x], first[x]) for x in first)
    t, ws = c.outputs(), c.workspace()
    other = Case(n, 4001, 136, k=k, seed=1)
    wanted = {x: y.clone() for x, y in other.check().items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(t, ws)
        c.grad(t, ws)
    names = ("hidden", "weight") + (("index", "teacher") if k else ("targets",))
    kept = {x: getattr(c, x).clone() for x in names}
    for values, want in ((kept, first), ({x: getattr(other, x) for x in names}, wanted),
                         (kept, first)):
        for x in names:
            getattr(c, x).copy_(values[x])
        ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t[x], want[x]) for x in want)


@pytest.mark.parametrize("k", [0, 5])
def test_gradients_against_differences(k):
    """The directional derivative of the loss in 64 bits, by central differences.
    The third derivative along a unit step in every logit is at most a few
    times the loss's weight: with steps of 2^-10 in directions whose logits
    move by up to 1 the differences are off by less than 2^-18 in all."""
    c = Case(60, 400, 64, k=k, tau=2.0 if k else 1.0, weighted=True)
    t = c.check()
    g = torch.Generator(device="cuda").manual_seed(3)
    args = (c.targets, c.index, c.teacher, c.tau, c.weights)
    for name in ("hidden", "weight"):
        x = getattr(c, name).double()
        u = torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64)
        y = (c.weight if name == "hidden" else c.hidden).double()
        u /= (u @ y.T).abs().max()                   # logits move by up to 1
        step = 2.0 ** -10

        def mean(sign):
            moved = x + sign * step * u
            pair = (moved, c.weight) if name == "hidden" else (c.hidden, moved)
            total = reference(*pair, *args)["total"][0]
            return float(total[0] / total[1])
        slope = (mean(1) - mean(-1)) / (2 * step)
        value, bound = c.reference()["d_" + name]
        got = float((t["d_" + name].double() * u).sum())
        assert abs(got - slope) <= float((bound * u.abs()).sum()) + 2.0 ** -18


@pytest.mark.parametrize("k", [0, 3])
def test_offsets_beyond_32_bits(k):
    """More logits than 2^31, in chunks of tokens against the reference."""
    n, v, d = 70001, 40009, 24
    assert n * v > 2 ** 31
    c = Case(n, v, d, k=k, weighted=True)
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    c.grad(t, ws, mean=False, scale=1e-3)
    torch.cuda.synchronize()
    weight, bound = (torch.zeros(v, d, dtype=torch.float64, device="cuda") for _ in range(2))
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    slack = torch.zeros(2, dtype=torch.float64, device="cuda")
    for first in range(0, n, 10000):
        rows = slice(first, min(n, first + 10000))
        part = [None if x is None else x[rows] for x in (c.targets, c.index, c.teacher)]
        ref = reference(c.hidden[rows], c.weight, *part, c.tau, c.weights[rows], scale=1e-3,
                        mean=False)
        assert outside({x: t[x][rows] for x in ("loss", "lse", "d_hidden")}, ref) == {}
        weight += ref["d_weight"][0]
        bound += ref["d_weight"][1]
        total += ref["total"][0]
        slack += ref["total"][1]
    assert outside(dict(d_weight=t["d_weight"], total=t["total"]),
                   dict(d_weight=(weight, bound), total=(total, slack))) == {}
    assert all(x.intact() for x in c.o.values())
