"""Tokens of weight 0 whose words lie beyond the vocabulary, as padding has them:
their loss is NaN, and they are out of total and of the gradients."""
import pytest
import torch

from head_reference import outside
from test_gpu_head import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 100, 300])
@pytest.mark.parametrize("k", [0, 4, 80])
@pytest.mark.parametrize("mean", [False, True])
def test_a_weight_of_0_takes_out_a_word_beyond_the_vocabulary(n, k, mean):
    c = Case(n, 301, 72, k=k, ignored=0.2, weighted=True)
    rows = torch.arange(0, n, 3, device="cuda")
    c.weights[rows] = 0.0
    (c.index[:, 0] if k else c.targets)[rows] = 5          # they count, with a weight of 0
    want = c.reference(mean=mean, scale=0.5)
    (c.index[:, 0] if k else c.targets)[rows] = 301
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    c.grad(t, ws, 0.5, mean)
    torch.cuda.synchronize()
    assert bool(t["loss"][rows].isnan().all())
    assert bool((t["d_hidden"][rows] == 0).all())
    for x in ("loss", "lse"):
        t[x][rows] = want[x][0][rows].float()
    assert outside(t, want) == {}
    assert all(x.intact() for x in c.o.values())
    # with a weight it is as before
    c.weights[rows[0]] = 1.0
    c.grad(t, ws, 0.5, mean)
    torch.cuda.synchronize()
    assert bool(t["d_weight"].isnan().all()) and bool(t["d_hidden"][rows[0]].isnan().all())
    assert bool((t["d_hidden"][rows[1:]] == 0).all())


@pytest.mark.parametrize("k", [0, 4])
def test_a_weight_of_0_beside_a_total_that_is_not_a_number(k):
    """Another token's loss and weight have spoilt the total: rows out of the
    gradients stay out of them."""
    c = Case(20, 301, 72, k=k, ignored=0.0, weighted=True)
    c.weights[3] = 0.0
    t, ws = c.outputs(), c.workspace()
    c.forward(t, ws)
    t["total"].fill_(float("nan"))
    c.grad(t, ws)
    torch.cuda.synchronize()
    assert bool((t["d_hidden"][3] == 0).all())
