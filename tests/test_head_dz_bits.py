"""The bounds of head_reference bind on the precision of dz: with the eight bits
of bf16 a plain form is inside, with fewer it is not.

dz enters two products, whose bound counts every term's half step as if all had one
sign.  Where one term makes nearly all of a sum, that is what the error comes to; so
with a word to each token, all different, some row of d_weight is one token's, and a
coarser dz shows there: with b bits it is off by up to 2^-b of the value, and the
bound, which has a half step for dz and one for the result, is about 2 x 2^-8."""
import pytest
import torch

from head_reference import outside, reference

N, V, D = 50, 300, 64


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) * D ** -0.5).to(torch.bfloat16)
    y = torch.randperm(V, generator=g)[:N]
    h = (torch.randn(N, D, generator=g) + 2 * w[y].float()).to(torch.bfloat16)
    y[::7] = -100
    return h, w, y


def rounded(x, bits):
    """To that many significant bits, to the nearest."""
    m, e = torch.frexp(x)
    return torch.ldexp((m * 2 ** bits).round() / 2 ** bits, e)


def form(h, w, y, bits):
    z = h.float() @ w.float().T
    lse = torch.logsumexp(z, dim=1)
    counts = y >= 0
    goal = torch.zeros_like(z)
    goal[counts, y[counts]] = 1.0
    a = counts.float()[:, None] / counts.sum()
    dz = rounded(a * (torch.exp(z - lse[:, None]) - goal), bits)
    return dict(d_hidden=(dz @ w.float()).to(torch.bfloat16),
                d_weight=(dz.T @ torch.where(counts[:, None], h.float(), 0.0)).to(torch.bfloat16))


@pytest.mark.parametrize("seed", range(4))
def test_eight_bits_are_inside(seed):
    args = inputs(seed)
    got = form(*args, 8)
    assert all(bool(x.isfinite().all()) for x in got.values())
    assert outside(got, reference(*args)) == {}


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("bits", [6, 5, 4])
def test_fewer_are_outside(seed, bits):
    args = inputs(seed)
    got = form(*args, bits)
    assert all(bool(x.isfinite().all()) for x in got.values())
    assert "d_weight" in outside(got, reference(*args))
