"""Plain 64-bit losses over a vocabulary with their gradients, and bounds on
what binary32 sums and roundings to bf16 may change of them.

Bounds.  u = 2^-24 is half a step of binary32, b = 2^-8 of bf16.
* A logit is a sum of `dim` exact products in binary32, in any order, each
  addition off by at most 2u (the tensor cores may cut off where others round):
  |dz| <= 2u (dim + 8) S with S = sum_c |hidden_c weight_c|.
* lse: the logits' error (a softmax mean of them, so at most their largest, over
  the temperature), then sums of at most vocab positive terms through chains of
  fewer than 2^9 additions, powers of two off by 2^-21, and the argument's
  rounding, 4u times its size: 2^-14 + 4u max |z| / tau.  loss: that of lse, of
  the logits, and of adding them up.
* p: the relative errors of both, as a factor exp(e) - 1.
* dz = a (p - q): a times the error of p and 8u (p + q) (q is computed in binary32
  too: 2^-18 q for its exponentials), then b of itself.
* a product of dz: the errors of its terms, 2u (terms + 8) of their absolute
  sum, and b of the result.
"""
import torch

U, B = 2.0 ** -24, 2.0 ** -8


def goal_of(targets, index, teacher, tau, n, v, device):
    """The distribution aimed at, its negative entropy, and which tokens count."""
    q = torch.zeros(n, v, dtype=torch.float64, device=device)
    if targets is not None:
        counts = targets >= 0
        rows = counts.nonzero()[:, 0]
        q[rows, targets[rows].long()] = 1.0
        return q, torch.zeros(n, dtype=torch.float64, device=device), counts
    x = teacher.double() / tau
    there = (index >= 0) & (teacher.double() != -torch.inf)
    counts = there.any(dim=1)
    x = torch.where(there, x, -torch.inf)
    x = torch.where(counts[:, None], x, 0.0)
    each = torch.where(there, torch.softmax(x, dim=1), 0.0)
    q.scatter_add_(1, index.long().clamp(min=0), each)
    return q, torch.where(each > 0, each * each.clamp(min=1e-300).log(), 0.0).sum(dim=1), counts


def reference(hidden, weight, targets=None, index=None, teacher=None, tau=1.0, weights=None,
              scale=1.0, mean=True):
    """{name: (value, bound)} of loss, lse, total, d_hidden and d_weight."""
    n, d = hidden.shape
    v = weight.shape[0]
    dev = hidden.device
    q, neg_entropy, counts = goal_of(targets, index, teacher, tau, n, v, dev)
    keep = counts[:, None]
    h = torch.where(keep, hidden.double(), 0.0)
    w = weight.double()
    z = h @ w.T
    size = (h.abs() @ w.abs().T)
    dlogit = 2 * U * (d + 8) * size
    zmax = dlogit.amax(dim=1) if n else dlogit.sum(dim=1)
    lse = torch.logsumexp(z / tau, dim=1)
    big = z.abs().amax(dim=1) / tau if n else lse
    dlse = zmax / tau + 2.0 ** -14 + 4 * U * (big + lse.abs())
    loss = tau * tau * (neg_entropy - (q * z).sum(dim=1) / tau + lse)
    # the terms q (log q - z / tau + lse), their errors and those of their sum
    parts = neg_entropy.abs() + (q * z.abs()).sum(dim=1) / tau + lse.abs() + 1
    dloss = tau * tau * (dlse + zmax / tau + 2.0 ** -16 * parts)
    if targets is not None:
        dloss = dlse + zmax + 4 * U * (lse.abs() + (q * z.abs()).sum(dim=1))
    each = (weights.double() if weights is not None
            else torch.ones(n, dtype=torch.float64, device=dev)) * counts
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    loss, lse_out = torch.where(counts, loss, zero), torch.where(counts, lse, zero)
    total = torch.stack([(each * loss).sum(), each.sum()])
    dtotal = torch.stack([(each.abs() * dloss).sum() + 2 * U * (each * loss).abs().sum(),
                          2 * U * each.abs().sum()])
    out = dict(loss=(loss, dloss), lse=(lse_out, dlse), total=(total, dtotal))
    a = scale * tau * each
    if mean:
        a = a / total[1] if float(total[1]) != 0 else a * 0
    p = torch.exp(z / tau - lse[:, None])
    dp = p * torch.expm1(dlogit / tau + dlse[:, None] + 4 * U * (z / tau).abs())
    dz = a[:, None] * (p - q)
    raw = a.abs()[:, None] * (dp + 8 * U * (p + q) + (0 if targets is not None else 2.0 ** -18) * q)
    ddz = raw + B * (dz.abs() + raw) + 2.0 ** -126
    for name, x, dx, y, terms in (("d_hidden", dz, ddz, w, v), ("d_weight", dz.T, ddz.T, h, n)):
        value = x @ y
        bound = dx @ y.abs() + 2 * U * (terms + 8) * ((x.abs() + dx) @ y.abs())
        out[name] = (value, bound + B * (value.abs() + bound) + 2.0 ** -126)
    return out


def outside(got, ref):
    """The names of the outputs that lie beyond their bounds, with the worst ratio."""
    bad = {}
    for name, x in got.items():
        if x is None:
            continue
        value, bound = ref[name]
        err = (x.double() - value).abs()
        ok = err <= bound                     # false for NaN
        if not bool(ok.all()):
            worst = torch.where(ok, 0.0, (err / bound).nan_to_num(nan=float("inf")))
            at = int(worst.argmax())
            bad[name] = (float(worst.max()), at, int((~ok).sum()), x.numel())
    return bad
