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


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("numel,ranks", [([35, 13, 12], 4), ([4096, 8192, 64], 8),
                                         ([100003, 7, 4099], 3)])
def test_halved_gradients_reduced_and_gathered(z3, ws, numel, ranks, graph):  # noqa: F811
    """The kernels that read bf16 with 16-byte loads right after a kernel of
    the library that wrote them: the reduce-scatters after a clipping of the
    ranks' gradients in place, the all-gather after a clipped update of the
    shards."""
    L = z3.Layout(numel, ranks)
    pitch = -(-L.psi // 8) * 8
    grads = normal(ranks * pitch, 1e4, B16, 3).view(ranks, pitch)
    tl = z3.TensorList([grads])
    out = torch.zeros(TURNS, 4, device="cuda")
    z3.z3_grad_norm(tl, 1.0, out[0, :2], ws)
    first = float(out[0, 0])
    T = -(-L.psi_padded // 8) * 8
    reduced = torch.zeros(2 * TURNS, T, device="cuda")
    sq = torch.zeros(TURNS, -(-L.sumsq_len // 2) * 2, dtype=torch.float64, device="cuda")
    z3.z3_reduce_scatter(L, grads, pitch, reduced[0, :L.psi_padded], 0.25)
    whole = reduced[0].clone()

    master, m, v, zero = (torch.zeros(L.psi_padded, device="cuda") for _ in range(4))
    master.copy_(normal(L.psi_padded, 1.0, F32, 4))
    shards = torch.empty(L.psi_padded, dtype=B16, device="cuda")
    full = torch.zeros(TURNS, pitch, dtype=B16, device="cuda")
    one = torch.tensor([1.0, 1.0], device="cuda")
    decay = dict(lr=0.5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=1.0)
    start = master.to(B16)
    z3.z3_allgather(L, start, full[0, :L.psi])
    gathered = full[0].clone()

    def chain():
        for i in range(TURNS):
            z3.z3_grad_norm(tl, first * 0.5 ** (i + 1), out[i, :2], ws)
            z3.z3_clip(tl, out[i, :2])
            z3.z3_reduce_scatter_norm(L, grads, pitch, reduced[2 * i, :L.psi_padded], 0.25,
                                      sq[i, :L.sumsq_len])
            z3.z3_reduce_scatter(L, grads, pitch, reduced[2 * i + 1, :L.psi_padded], 0.25)
            # no gradient: p <- p - lr * weight_decay * p = p / 2
            z3.z3_adam_shard_step_clipped(L, master, m, v, zero, shards, decay, 1, one)
            z3.z3_allgather(L, shards, full[i, :L.psi])
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain()
        g.replay()
    else:
        chain()
    for i in range(TURNS):
        assert torch.equal(reduced[2 * i], whole * 0.5 ** (i + 1)), i
        assert torch.equal(reduced[2 * i + 1], whole * 0.5 ** (i + 1)), i
        assert torch.equal(full[i], gathered * 0.5 ** (i + 1)), i
    total = sq[:, :L.sumsq_len].sum(1).tolist()
    assert total == [total[0] * 0.25 ** i for i in range(TURNS)]
