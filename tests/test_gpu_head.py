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
