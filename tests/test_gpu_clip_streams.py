"""Clipped model steps on other streams than the current one, bit for bit
against steps on the current stream."""
import pytest
import torch

from test_gpu_clip import HP, make_model, model_bits, same, z3  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


def keep_busy():
    """Some 50 ms of work on the current stream."""
    x = torch.zeros(1 << 28, device="cuda")
    for _ in range(150):
        x.add_(1.0)
    return x


def everything(m):
    bits = model_bits(m)                          # waits for the device
    return bits, m.clip.clone(), [(g.clone(), s.clone()) for g, s in m.clip_args()]


def assert_same(got, want):
    assert same(got[0], want[0]) and torch.equal(got[1], want[1])
    for (g, s), (h, t) in zip(got[2], want[2]):
        assert torch.equal(g, h) and torch.equal(s, t)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("prefetch", [0, 1])
def test_first_clipped_step_on_a_side_stream(z3, prefetch, hooked, handle):  # noqa: F811
    """The current stream is busy while the side stream takes the first
    clipped step: nothing that the step allocates may wait behind that work
    and land on top of the step's results."""
    hook = {"on_gather": lambda *a: None} if hooked else {}
    a, b = make_model(prefetch, (1,)), make_model(prefetch, (1,))
    a.step(HP, max_norm=0.01, **hook)
    want = everything(a)
    assert 0 < float(want[1][1]) < 1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = keep_busy()
    b.step(HP, stream=side.cuda_stream if handle else side, max_norm=0.01, **hook)
    assert_same(everything(b), want)
    del busy


def test_buffers_asked_for_on_a_busy_stream(z3):  # noqa: F811
    a, b = make_model(0), make_model(0)
    a.step(HP, max_norm=0.01)
    want = everything(a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = keep_busy()
    b.clip_args()
    b.step(HP, stream=side, max_norm=0.01)
    assert_same(everything(b), want)
    del busy


def test_first_clipped_step_inside_a_capture(z3):  # noqa: F811
    """Its buffers are of the graph's memory; a later step may use them too."""
    a, b = make_model(0), make_model(0)
    for t in (1, 2):
        a.step(HP, t=t, max_norm=0.01)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step(HP, t=1, max_norm=0.01)
    g.replay()
    b.step(HP, t=2, max_norm=0.01)
    assert_same(everything(b), everything(a))
