"""Which stream a clipped model step allocates on, on the CPU: torch's allocator
and fills, the streams and the library's calls are replaced by recorders.

What a clipped step allocates for itself is filled and handed out in the order
of one stream; kernels on another stream would run before, beside or after
those fills.  So the step's own stream has to be the one, or wait for it."""
import contextlib
import itertools
import types

import pytest
import torch

from optimizer_state_gb300 import schedule


class Stream:
    handles = itertools.count(1)

    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, next(self.handles)

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))

    def wait_event(self, event):
        pass


class Recorder:
    """Replaces what schedule uses of torch.cuda and the library by a log of
    ("alloc", stream), ("wait", stream, for stream) and ("call", name, stream)."""

    def __init__(self, monkeypatch):
        self.log = []
        self.current = self.default = Stream("default", self.log)
        self.streams = {s.cuda_stream: s for s in [self.default]}
        self.capturing = set()
        cuda = torch.cuda
        monkeypatch.setattr(cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(cuda, "default_stream", lambda *a: self.default)
        monkeypatch.setattr(cuda, "ExternalStream", lambda h: self.streams[h])
        monkeypatch.setattr(cuda, "Stream", lambda **k: self.stream("gather"))
        monkeypatch.setattr(cuda, "Event", lambda: types.SimpleNamespace(record=lambda s: None))
        monkeypatch.setattr(cuda, "stream", self.under)
        monkeypatch.setattr(cuda, "is_current_stream_capturing",
                            lambda: self.current.name in self.capturing)
        for name in ("zeros", "empty"):
            monkeypatch.setattr(torch, name, self.allocating(getattr(torch, name)))
        monkeypatch.setattr(schedule, "z3", types.SimpleNamespace(
            TensorList=lambda *a, **k: None, grad_norm_workspace=self.workspace,
            **{n: self.call(n) for n in (
                "z3_model_step", "z3_model_step_clipped", "z3_allgather", "z3_grad_norm",
                "z3_reduce_scatter_norm", "z3_reduce_scatter_adam",
                "z3_adam_shard_step_clipped")}))

    def stream(self, name):
        s = Stream(name, self.log)
        self.streams[s.cuda_stream] = s
        return s

    @contextlib.contextmanager
    def under(self, s):
        kept, self.current = self.current, s
        try:
            yield
        finally:
            self.current = kept

    def allocating(self, real):
        def alloc(*a, **k):
            self.log.append(("alloc", self.current.name))
            return real(*a, **{**k, "device": "cpu"})
        return alloc

    def workspace(self, device):
        self.log.append(("alloc", self.current.name))
        return None

    def call(self, name):
        def f(*a, stream=None, gather_stream=None):
            if stream is None:
                s = self.current
            elif isinstance(stream, int):
                s = self.default if stream == 0 else self.streams[stream]
            else:
                s = stream
            self.log.append(("call", name, s.name))
        return f


CLIPPING = ("z3_model_step_clipped", "z3_grad_norm", "z3_reduce_scatter_norm",
            "z3_adam_shard_step_clipped")


def unordered(log):
    """The calls that use a clipped step's buffers on a stream that is neither
    the one they were allocated on nor has waited for it."""
    seen, bad = set(), []       # (stream, allocating stream it knows of)
    owners = set()
    for e in log:
        if e[0] == "alloc":
            owners.add(e[1])
            seen = {x for x in seen if x[1] != e[1]} | {(e[1], e[1])}
        elif e[0] == "wait":
            seen |= {(e[1], o) for s, o in seen if s == e[2]}
        elif e[1] in CLIPPING:
            bad += [e for o in owners if (e[2], o) not in seen]
    return bad


@pytest.fixture()
def rec(monkeypatch):
    return Recorder(monkeypatch)


def make(rec, prefetch):
    L = types.SimpleNamespace(psi=6, psi_padded=8, sumsq_len=1, n_ranks=2, numel=[6])
    unit = types.SimpleNamespace(
        L=L, shards=None, master=None, m=None, v=None, grads=None, resident=None, hp=None,
        w=types.SimpleNamespace(grad_stride=8, n_ranks=2))
    model = schedule.PrefetchModel([unit, unit], "cpu", 1) if prefetch else \
        schedule.Model([unit, unit], "cpu")
    rec.log.clear()
    return model


@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("prefetch", [False, True])
@pytest.mark.parametrize("given", ["none", "stream", "handle", "zero"])
def test_first_clipped_step_allocates_in_its_streams_order(rec, prefetch, given, hooked):
    model, side = make(rec, prefetch), rec.stream("side")
    if given == "zero":          # handle 0 is the default stream, whatever is current
        rec.current = side
    stream = {"none": None, "stream": side, "handle": side.cuda_stream, "zero": 0}[given]
    hook = {"on_gather": lambda *a: None} if hooked else {}
    for _ in range(2):
        model.step({}, stream=stream, max_norm=1.0, **hook)
    assert any(e[0] == "alloc" for e in rec.log)
    assert any(e[0] == "call" and e[1] in CLIPPING for e in rec.log)
    assert unordered(rec.log) == []
    n = sum(e[0] == "alloc" for e in rec.log)
    model.step({}, stream=stream, max_norm=1.0, **hook)
    assert sum(e[0] == "alloc" for e in rec.log) == n       # once


@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("prefetch", [False, True])
def test_a_step_waits_for_buffers_that_were_asked_for_elsewhere(rec, prefetch, hooked):
    model, side = make(rec, prefetch), rec.stream("side")
    hook = {"on_gather": lambda *a: None} if hooked else {}
    model.clip_args()                                       # on the current stream
    model.step({}, stream=side, max_norm=1.0, **hook)
    assert unordered(rec.log) == []


def test_a_captured_step_waits_for_nothing_outside_its_capture(rec):
    """A wait for work outside a capture cannot be captured; the next step
    that is not captured still waits."""
    model, graph, side = make(rec, False), rec.stream("graph"), rec.stream("side")
    model.clip_args()
    rec.capturing.add("graph")
    model.step({}, stream=graph, max_norm=1.0)
    assert not any(e[0] == "wait" for e in rec.log)
    rec.log.clear()
    rec.log.append(("alloc", "default"))
    model.step({}, stream=side, max_norm=1.0)
    assert unordered(rec.log) == []


def test_a_step_that_is_not_clipped_allocates_nothing(rec):
    model, side = make(rec, False), rec.stream("side")
    model.step({}, stream=side)
    model.step({}, stream=side, on_gather=lambda *a: None)
    assert not any(e[0] == "alloc" for e in rec.log) and model.clip is None
