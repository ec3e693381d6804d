"""A head's buffers on other streams than the one that they were allocated on, on
the CPU: torch's streams and allocator and the library's calls are replaced by
recorders.

A freed buffer goes back to the stream that it was allocated on at once, unless the
allocator was told who else uses it.  Kernels that still run on another stream
would then write into what is another tensor's by now."""
import contextlib
import types

import pytest
import torch

from optimizer_state_gb300 import schedule

RANKS, TOKENS, VOCAB, DIM = 2, 3, 16, 8


class Fakes:
    def __init__(self, monkeypatch):
        def stream(handle):
            return types.SimpleNamespace(cuda_stream=handle, wait_stream=self.waits.append)
        self.waits, self.capturing, self.recorded = [], False, {}
        self.streams = {h: stream(h) for h in (1, 2, 3)}
        cuda = torch.cuda
        monkeypatch.setattr(cuda, "current_stream", lambda *a: self.streams[1])
        monkeypatch.setattr(cuda, "default_stream", lambda *a: self.streams[1])
        monkeypatch.setattr(cuda, "ExternalStream", lambda h: self.streams[h])
        monkeypatch.setattr(cuda, "stream", lambda s: contextlib.nullcontext())
        monkeypatch.setattr(cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: self.record(x, s))
        none = {n: (lambda *a, **k: None) for n in ("z3_allgather", "z3_xent", "z3_xent_grad")}
        monkeypatch.setattr(schedule, "z3", types.SimpleNamespace(
            head_workspace=lambda *a: torch.empty(64, dtype=torch.uint8), **none))
        psi = VOCAB * DIM
        unit = types.SimpleNamespace(
            L=types.SimpleNamespace(psi=psi, full_off=[0]), resident=None, shards=None,
            w=types.SimpleNamespace(shapes=((VOCAB, DIM),), n_ranks=RANKS),
            grads=torch.zeros(RANKS, psi, dtype=torch.bfloat16))
        model = types.SimpleNamespace(units=[unit], dev="cpu",
                                      full=torch.zeros(psi, dtype=torch.bfloat16))
        self.head = schedule.Head(model, TOKENS)
        self.hidden = torch.zeros(RANKS, TOKENS, DIM, dtype=torch.bfloat16)
        self.targets = torch.zeros(RANKS, TOKENS, dtype=torch.long)

    def record(self, tensor, stream):
        at = tensor.untyped_storage().data_ptr()
        self.recorded.setdefault(stream.cuda_stream, set()).add(at)

    def call(self, stream):
        self.head(self.hidden, self.targets, stream=stream)

    def buffers(self):
        """Whatever tensors the head itself holds."""
        return {x.untyped_storage().data_ptr() for x in vars(self.head).values()
                if isinstance(x, torch.Tensor)}


@pytest.mark.parametrize("captured", [False, True])
def test_every_buffer_is_recorded_on_every_stream_that_uses_it(monkeypatch, captured):
    f = Fakes(monkeypatch)
    f.capturing = captured
    assert len(f.buffers()) == 5
    for s in (2, 3, 2):
        f.call(f.streams[s])
    assert f.recorded == {2: f.buffers(), 3: f.buffers()}


def test_not_on_their_own(monkeypatch):
    f = Fakes(monkeypatch)
    f.call(None)
    f.call(f.streams[1])
    f.call(0)                                           # the default stream's handle
    assert f.recorded == {} and f.waits == []


def test_a_raw_handle_is_the_callers(monkeypatch):
    """Its stream may be gone when the buffers are freed: nothing is asked of it then."""
    f = Fakes(monkeypatch)
    f.call(2)
    assert f.recorded == {} and f.waits == [f.streams[1]]
    f.call(f.streams[3])
    assert f.recorded == {3: f.buffers()}


def test_the_first_call_waits_once(monkeypatch):
    f = Fakes(monkeypatch)
    f.capturing = True
    f.call(f.streams[2])
    assert f.waits == []                                # left to the next
    f.capturing = False
    f.call(f.streams[2])
    f.call(f.streams[2])
    assert f.waits == [f.streams[1]]


@pytest.mark.gpu
def test_a_head_that_goes_before_its_calls_end():
    """Its memory is not handed out while a side stream still uses it."""
    from optimizer_state_gb300 import build, inputs, schedule as sch, z3
    build.build()
    z3.load()
    dev = torch.device("cuda")
    unit = sch.Unit(inputs.Workload("embed", ((1003, 64),), RANKS, 0.02, 1e-3), dev,
                    inputs.make_generator(3, dev))
    model = sch.Model([unit], dev)
    head = model.head(40)
    hidden = torch.zeros(RANKS, 40, 64, dtype=torch.bfloat16, device=dev)
    targets = torch.zeros(RANKS, 40, dtype=torch.long, device=dev)
    model.head(40)(hidden, targets)                     # its kernels are loaded
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1 << 28)                      # an eighth of a second
        head(hidden, targets)
    places = {x.data_ptr(): x.numel() * x.element_size() for x in vars(head).values()
              if isinstance(x, torch.Tensor)}
    del head
    taken = [torch.empty(n, dtype=torch.uint8, device=dev) for n in places.values()]
    assert not side.query()                             # the calls have not ended
    assert all(x.data_ptr() not in places for x in taken)
    torch.cuda.synchronize()
