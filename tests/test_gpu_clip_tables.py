"""Tensor lists beside the sizes of the launch tables, which fill 4, 8 and 16 KB
and 32,764 bytes of kernel parameters: a table of c tensors takes a head of
1,048 bytes and c + 1 entries of 16, beside 32 bytes for the other argument."""
import pytest
import torch

from test_gpu_clip import (B16, F32, back_to_back, check_norm, clip,  # noqa: F401
                           exact_norm, ws, z3)

pytestmark = pytest.mark.gpu

FULL = [(b - 1048 - 32) // 16 - 1 for b in (4096, 8192, 16384, 32764)]


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("count", [c + d for c in FULL for d in (-1, 0, 1)] +
                         [2 * FULL[-1], 2 * FULL[-1] + 1])
def test_counts_beside_the_tables_sizes(z3, clip, ws, count, dtype):  # noqa: F811
    buf, views = back_to_back([5 + 31 * (i % 3) for i in range(count)], dtype, 1e-3, count,
                              shift=3)
    before = buf.t.clone()
    want = exact_norm([buf.t[3:]])
    tl = z3.TensorList(views)
    z3.z3_grad_norm(tl, 0.37 * want, clip, ws)
    check_norm(clip, want, 0.37 * want)
    z3.z3_clip(tl, clip)
    scaled = (before.float() * clip[1]).to(dtype)
    scaled[:3] = before[:3]
    assert torch.equal(buf.t, scaled) and buf.guards_intact()
    # what the last tensor holds is seen, and no more than the list
    views[-1][-1] = float("nan")
    z3.z3_grad_norm(tl, 1.0, clip, ws)
    assert clip.isnan().all()
    z3.z3_grad_norm(views[:-1], 1.0, clip, ws)
    check_norm(clip, exact_norm(views[:-1]), 1.0)
