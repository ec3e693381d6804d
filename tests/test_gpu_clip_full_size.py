"""The clipped kernels at full size: positions beyond 32 bits, the d = 4096
layer, and the 24-layer model, on every schedule.

The large layers are compared whole and bit for bit with the kernels of the
step that is not clipped (tested against the oracle at these sizes
elsewhere): the reduced gradient with z3_reduce_scatter's, the update with
z3_adam_shard_step's on coef * gradient in binary32.  Norms are compared with
64-bit sums at 2^-21, the bound of 13 roundings below them."""
import math

import numpy as np
import pytest
import torch

from test_gpu_clip import B16, F32, HP, clip, normal, ws, z3  # noqa: F401
from optimizer_state_gb300 import inputs as I

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -21


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def squares(t):
    return sum(float(p.double().square().sum()) for p in t.split(1 << 28))


def bits_equal(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == B16 else torch.int32),
                       b.view(torch.int16 if b.dtype == B16 else torch.int32))


def test_positions_beyond_32_bits(z3, orc, clip, ws):  # noqa: F811
    """One parameter of 2^32 + 11 elements over 2 ranks, zero but at positions
    beside every power of two that an index could be cut at."""
    n, ranks = 2 ** 32 + 11, 2
    L = z3.Layout([n], ranks)
    pitch = -(-n // 8) * 8
    s = L.psi_padded // ranks
    places = [0, 1, 2 ** 31 - 1, 2 ** 31, s - 1, s, 2 ** 32 - 1, 2 ** 32, n - 1]
    grads = torch.zeros(ranks * pitch, dtype=B16, device="cuda")
    for i, x in enumerate(places):
        grads[x] = i + 1.0
        grads[pitch + x] = 0.5
    out = torch.full((L.psi_padded,), math.nan, device="cuda")
    sq = torch.empty(L.sumsq_len, dtype=torch.float64, device="cuda")
    z3.z3_reduce_scatter_norm(L, grads, pitch, out, 0.5, sq)
    assert int(out.count_nonzero()) == len(places)
    values = [0.5 * (i + 1.5) for i in range(len(places))]
    assert [float(out[x]) for x in places] == values        # one parameter: no gaps
    z3.z3_reduce_scatter_norm(L, grads, pitch, out, 0.5, sq, accumulate=True)
    assert int(out.count_nonzero()) == len(places)
    values = [2 * v for v in values]
    assert [float(out[x]) for x in places] == values
    assert float(sq.sum()) == sum(v * v for v in values)
    z3.z3_grad_norm(z3.TensorList([], sumsq=[sq]), 1.0, clip, ws)
    want = math.sqrt(sum(v * v for v in values))
    assert abs(float(clip[0].double()) - want) <= TOL * want
    del grads, sq

    master, m, v = (torch.zeros(L.psi_padded, device="cuda") for _ in range(3))
    shards = torch.ones(L.psi_padded, dtype=B16, device="cuda")
    z3.z3_adam_shard_step_clipped(L, master, m, v, out, shards, HP, 3, clip)
    g = np.array(values, np.float32) * np.float32(float(clip[1]))
    p, hm, hv = (np.zeros(len(places), np.float32) for _ in range(3))
    bf = np.zeros(len(places), np.uint16)
    orc.adam(p, hm, hv, g, bf, HP["lr"], HP["beta1"], HP["beta2"], HP["eps"],
             HP["weight_decay"], 3)
    for t, h in ((master, p), (m, hm), (v, hv)):
        assert int(t.count_nonzero()) == len(places)
        assert [float(t[x]) for x in places] == h.tolist()
    assert int(shards.count_nonzero()) == len(places)
    assert [int(shards[x].view(torch.int16)) & 0xffff for x in places] == bf.tolist()


@pytest.mark.parametrize("ranks", [8, 64])
def test_d4096_layer(z3, clip, ws, ranks):  # noqa: F811
    w = I.layer_7b(ranks)
    L = z3.Layout(w.numel, w.n_ranks)
    T, scale = L.psi_padded, 1.0 / w.n_ranks
    grads = I.draw_grads(w, I.make_generator(5, "cuda"), "cuda")
    want, got = (torch.full((T,), math.nan, device="cuda") for _ in range(2))
    sq = torch.empty(L.sumsq_len, dtype=torch.float64, device="cuda")
    z3.z3_reduce_scatter(L, grads, w.grad_stride, want, scale)
    z3.z3_reduce_scatter_norm(L, grads, w.grad_stride, got, scale, sq)
    assert bits_equal(got, want)
    z3.z3_reduce_scatter(L, grads, w.grad_stride, want, scale, accumulate=True)
    z3.z3_reduce_scatter_norm(L, grads, w.grad_stride, got, scale, sq, accumulate=True)
    assert bits_equal(got, want)
    del grads
    norm = math.sqrt(squares(got))
    z3.z3_grad_norm(z3.TensorList([], sumsq=[sq]), 0.37 * norm, clip, ws)
    assert abs(float(clip[0].double()) - norm) <= TOL * norm

    a = [normal(T, 0.02, F32, 1), normal(T, 1e-3, F32, 2), normal(T, 1e-3, F32, 3).square_()]
    b = [t.clone() for t in a]
    sa, sb = (torch.empty(T, dtype=B16, device="cuda") for _ in range(2))
    z3.z3_adam_shard_step(L, *a, got * clip[1], sa, HP, 4)
    z3.z3_adam_shard_step_clipped(L, *b, got, sb, HP, 4, clip)
    assert bits_equal(got, want)
    for x, y in zip([*a, sa], [*b, sb]):
        assert bits_equal(x, y)


@pytest.mark.parametrize("prefetch,bucket,persist,hooked", [
    (0, 1, 0, False), (2, 4, 100000, False), (0, 6, 0, True), (1, 1, 0, True)])
def test_24_layer_model(z3, prefetch, bucket, persist, hooked):  # noqa: F811
    """The [50257, 1024] embedding and 24 layers over 16 ranks, two steps, one
    of them clipped."""
    from optimizer_state_gb300 import schedule
    m = schedule.full_step_model(torch.device("cuda"), 3, prefetch=prefetch,
                                 bucket_layers=bucket, persistence_threshold=persist)
    state = [[u.master.clone(), u.m.clone(), u.v.clone()] for u in m.units]
    reduced = [torch.empty(u.L.psi_padded, device="cuda") for u in m.units]
    for u, r in zip(m.units, reduced):
        z3.z3_reduce_scatter(u.L, u.grads, u.w.grad_stride, r, 1.0 / u.w.n_ranks)
    norm = math.sqrt(sum(squares(r) for r in reduced))
    hook = {"on_gather": lambda *a: None} if hooked else {}
    for t, max_norm in ((1, 0.37 * norm), (2, 2 * norm)):
        m.step(HP, max_norm=max_norm, **hook)
        assert abs(float(m.clip[0].double()) - norm) <= TOL * norm
        assert (float(m.clip[1]) < 1) == (t == 1)
        for u, s, r, (gs, _) in zip(m.units, state, reduced, m.clip_args()):
            assert bits_equal(gs, r)
            bf = torch.empty(u.L.psi_padded, dtype=B16, device="cuda")
            z3.z3_adam_shard_step(u.L, *s, r * m.clip[1], bf, HP, t)
            for x, y in zip([*s, bf], [u.master, u.m, u.v, u.shards]):
                assert bits_equal(x, y)
            if u.resident is not None:
                full = torch.empty_like(u.resident)
                z3.z3_allgather(u.L, u.shards, full)
                assert bits_equal(full, u.resident)
