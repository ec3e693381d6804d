"""A step whose loss raises, on the CPU: it has not taken place."""
import types

import pytest
import torch

from optimizer_state_gb300 import schedule

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)


class Steps:
    """A model of two units whose library calls are recorded."""

    def __init__(self, monkeypatch, prefetch):
        self.numbers = []

        def call(*a, **k):
            self.numbers.append(next(x for x in reversed(a) if isinstance(x, int)))
        monkeypatch.setattr(schedule, "z3", types.SimpleNamespace(
            z3_model_step=call, z3_reduce_scatter_adam=call, z3_allgather=lambda *a, **k: None))
        cuda = torch.cuda
        stream = types.SimpleNamespace(cuda_stream=1, wait_stream=lambda s: None,
                                       wait_event=lambda e: None)
        monkeypatch.setattr(cuda, "Stream", lambda **k: stream)
        monkeypatch.setattr(cuda, "current_stream", lambda *a: stream)
        monkeypatch.setattr(cuda, "Event", lambda: types.SimpleNamespace(record=lambda s: None))
        monkeypatch.setattr(cuda, "stream", lambda s: _Nothing())
        unit = types.SimpleNamespace(
            L=types.SimpleNamespace(psi=8), resident=None, shards=None, master=None, m=None, v=None,
            grads=None, hp=None, w=types.SimpleNamespace(grad_stride=8, n_ranks=2))
        units = [unit, unit]
        self.model = (schedule.PrefetchModel(units, "cpu") if prefetch
                      else schedule.Model(units, "cpu"))


class _Nothing:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


def bad(stream):
    raise ValueError("targets: needs shape")


@pytest.mark.parametrize("prefetch", [False, True])
@pytest.mark.parametrize("hooked", [False, True])
def test_it_keeps_no_number(monkeypatch, prefetch, hooked):
    s = Steps(monkeypatch, prefetch)
    how = dict(on_gather=lambda phase, i: None) if hooked else {}
    for number in (1, 2):
        with pytest.raises(ValueError, match="targets"):
            s.model.step(HP, loss=bad, **how)
        assert s.numbers == [] and s.model.t == number - 1
        s.model.step(HP, loss=lambda stream: None, **how)
        assert set(s.numbers) == {number} and s.model.t == number
        s.numbers.clear()
    # a caller's own number is the caller's
    with pytest.raises(ValueError, match="targets"):
        s.model.step(HP, t=9, loss=bad, **how)
    assert s.model.t == 2
