"""The bounds of head_reference hold for a plain form in 32 bits with dz rounded
to bf16, and bind: forms with a mistake planted in them lie outside."""
import pytest
import torch

from head_reference import outside, reference

N, V, D, K = 50, 300, 64, 6


def inputs(k, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) * D ** -0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g)
    h = (torch.randn(N, D, generator=g) + 6 * torch.rand(N, 1, generator=g) *
         w[y].float()).to(torch.bfloat16)
    weights = torch.rand(N, generator=g) + 0.25
    y[torch.rand(N, generator=g) < 0.2] = -100
    idx = torch.randint(0, V, (N, K), generator=g)
    idx[:, 5] = idx[:, 0]                            # a word twice
    idx[torch.rand(N, K, generator=g) < 0.1] = -1
    idx[3] = -1
    t = torch.randn(N, K, generator=g) * 2
    return (h, w, None, idx, t, 2.0, weights) if k else (h, w, y, None, None, 1.0, weights)


def form(h, w, y, idx, t, tau, weights, scale, wrong=None):
    """In binary32, as the kernels: dz rounded to bf16, results rounded once."""
    z = h.float() @ w.float().T
    if wrong == "temperature":
        tau = 1.0
    lse = torch.logsumexp(z / tau, dim=1)
    q = torch.zeros_like(z)
    if y is not None:
        counts = y >= 0
        q[counts, y[counts]] = 1.0
        neg = torch.zeros(N)
    else:
        there = idx >= 0
        counts = there.any(dim=1)
        x = torch.where(there, t / tau, -torch.inf)
        each = torch.where(there, torch.softmax(torch.where(counts[:, None], x, 0.0), dim=1), 0.0)
        if wrong == "same word once":
            q.scatter_(1, idx.clamp(min=0), each)
        else:
            q.scatter_add_(1, idx.clamp(min=0), each)
        neg = torch.where(each > 0, each * each.clamp(min=1e-30).log(), 0.0).sum(dim=1)
    power = tau if wrong == "tau once" else tau * tau
    loss = power * (neg - (q * z).sum(dim=1) / tau + lse)
    if wrong == "no entropy":
        loss = loss - power * neg
    if wrong == "loss off by 2^-8":
        loss = loss * (1 + 2.0 ** -8)
    a = scale * tau * weights * counts
    if wrong == "weights dropped":
        a = scale * tau * counts
    if wrong == "tau dropped":
        a = a / tau
    each = (weights if wrong != "weights dropped" else torch.ones(N)) * counts
    total = torch.stack([(each * loss).sum(), each.sum()])
    if wrong == "mean over all":
        total[1] = weights.sum()
    a = a / total[1]
    p = torch.exp(z / tau - lse[:, None])
    if wrong == "no target":
        q = q * 0
    if wrong == "target's neighbour":
        q = q.roll(1, dims=1)
    if wrong == "left out rows count":
        a = scale * tau * weights / total[1]
    dz = (a[:, None] * (p - q)).to(torch.bfloat16).float()
    if wrong == "dz in 7 bits":
        dz = (dz * 2 ** 20).to(torch.float8_e4m3fn).float() / 2 ** 20
    if wrong == "last word dropped":
        dz[:, -1] = 0
    out = dict(loss=torch.where(counts, loss, 0.0), lse=torch.where(counts, lse, 0.0), total=total,
               d_hidden=(dz @ w.float()).to(torch.bfloat16),
               d_weight=(dz.T @ torch.where(counts[:, None], h.float(), 0.0)).to(torch.bfloat16))
    if wrong == "d_weight of hidden's neighbour":
        out["d_weight"] = out["d_weight"].roll(1, dims=1)
    return out


@pytest.mark.parametrize("k", [0, K])
@pytest.mark.parametrize("seed", range(4))
def test_a_form_without_mistakes_is_inside(k, seed):
    args = inputs(k, seed)
    assert outside(form(*args, 0.5), reference(*args, scale=0.5)) == {}


BOTH = ("weights dropped", "mean over all", "no target", "target's neighbour",
        "left out rows count", "last word dropped", "d_weight of hidden's neighbour",
        "loss off by 2^-8")


@pytest.mark.parametrize("k,wrong", [(k, x) for k in (0, K) for x in BOTH] + [
    (K, x) for x in ("temperature", "tau once", "tau dropped", "no entropy", "same word once")])
def test_a_mistake_is_outside(k, wrong):
    args = inputs(k)
    assert outside(form(*args, 0.5, wrong), reference(*args, scale=0.5)) != {}
