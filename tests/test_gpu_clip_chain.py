"""Norm and clipping in turn, bit for bit: every call must see all that the one
before it wrote.

With max_norm half of the norm, coef is exactly 1/2.  Halving is exact in both
types (the values stay normal numbers), and each operation of a norm of halved
values gives the halved result (the sums a quarter): the i-th norm is the
first times 2^-i bit for bit.  A vector (4 or 8 of at most 2^21 elements) that
a norm read before the clipping had written it would move the sum by 3 * 4 /
2^21 of itself, some 2^-17, against the 2^-24 of a binary32 norm."""
import pytest
import torch

from test_gpu_clip import B16, F32, back_to_back, clip, normal, ws, z3  # noqa: F401

pytestmark = pytest.mark.gpu

TURNS = 40


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("lengths", [[7], [5000, 3], [17] * 300, [100003, 65537], [4099] * 200,
                                     [3, 1000003, 250007], [1 << 21]],
                         ids=lambda x: f"{len(x)}x{max(x)}")
def test_halving(z3, ws, lengths, graph, dtype):  # noqa: F811
    buf, views = back_to_back(lengths, dtype, 1e4, 8, shift=1)
    tl = z3.TensorList(views)
    out = torch.zeros(TURNS, 4, device="cuda")
    z3.z3_grad_norm(tl, 1.0, out[0, :2], ws)
    first = float(out[0, 0])
    before = buf.t.clone()

    def chain():
        for i in range(TURNS):
            z3.z3_grad_norm(tl, first * 0.5 ** (i + 1), out[i, :2], ws)
            z3.z3_clip(tl, out[i, :2])
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain()
        g.replay()
    else:
        chain()
    assert out[:, 0].tolist() == [first * 0.5 ** i for i in range(TURNS)]
    assert out[:, 1].tolist() == [0.5] * TURNS
    assert torch.equal(buf.t[1:], before[1:] * 0.5 ** TURNS)
    assert buf.guards_intact()
