"""The norm's precision where its roundings do not average out: equal values.

At most 13 binary32 roundings lie on a square's way into its batch (24
elements of a thread: 12 multiply-adds and an addition) or its warp (8
multiply-adds and 5 additions), each within u = 2^-24 of a sum of positive
terms: 13 u.  Batches are then added in pairs of binary32, which adds n^2 u^2 / 2
for n batches in one thread (under u / 2 for n < 4096).  The square root
halves the sum's relative error and the result is rounded once more:
(13 u + u / 2) / 2 + u = 7.75 u < 2^-21."""
import math

import numpy as np
import pytest
import torch

from test_gpu_clip import B16, F32, clip, ws, z3  # noqa: F401

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -21
# values whose squares round up, or down, time after time
VALUES = [1.7897, 1.2768, math.sqrt(2.0), 1.0 + 2.0 ** -12, 1.0 + 2.0 ** -23, 1.9999999, 1e-3]


def check(clip, want):  # noqa: F811
    norm = float(clip[0].double())
    assert abs(norm - want) <= TOL * want, (norm, want, (norm / want - 1) / TOL)


@pytest.mark.parametrize("n", [5, 24, 12288, 100003, 1 << 22])
@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("value", VALUES)
def test_norm_of_equal_values(z3, clip, ws, value, dtype, n):  # noqa: F811
    t = torch.full((n,), value, dtype=dtype, device="cuda")
    z3.z3_grad_norm([t], 1.0, clip, ws)
    check(clip, float(t[0].double()) * math.sqrt(n))


def test_norm_of_many_batches_per_thread(z3, clip, ws):  # noqa: F811
    n = (1 << 30) + 3                       # 4.3 GB: 384 batches
    t = torch.full((n,), 1.7897, device="cuda")
    z3.z3_grad_norm([t], 1.0, clip, ws)
    check(clip, float(np.float32(1.7897)) * math.sqrt(n))


@pytest.mark.parametrize("numel,ranks", [([12288 * 8], 8), ([4096, 8192, 64], 8),
                                         ([100003, 7, 4099], 3), ([1 << 22], 1)])
@pytest.mark.parametrize("value", VALUES)
def test_reduced_gradients_of_equal_values(z3, clip, ws, value, numel, ranks):  # noqa: F811
    L = z3.Layout(numel, ranks)
    pitch = -(-L.psi // 8) * 8
    grads = torch.ones(ranks * pitch, dtype=B16, device="cuda")
    out = torch.empty(L.psi_padded, device="cuda")
    sq = torch.empty(L.sumsq_len, dtype=torch.float64, device="cuda")
    z3.z3_reduce_scatter_norm(L, grads, pitch, out, value / ranks, sq)
    each = float(np.float32(ranks) * np.float32(value / ranks))
    assert int((out == each).sum()) == L.psi and int(out.count_nonzero()) == L.psi
    z3.z3_grad_norm(z3.TensorList([], sumsq=[sq]), 1.0, clip, ws)
    check(clip, each * math.sqrt(L.psi))
