"""Cross entropy of likely targets: the loss keeps its digits, and dz at the target
those that lse leaves it.

The inputs.  A token's logits are 16 and a little for its target, and for the other
V - 1 words the product of two bf16 values, exact in binary32 however it is
summed.  So all that can go wrong is the target's logit z, and what is made of it.
Its row is a term of 16, then D terms of 2^-20 to 2^-17, all positive: sums that cut off lose
about half a unit of 16, 2^-20, whenever some terms join the larger one.  (The places that would meet the large term in its
own chain of sums hold zeros, so that rounding has its say only where chains meet.)

Bounds.  With R = sum over the other words of exp(z_j - z), loss = log(1 + R) and
dz = -a R / (1 + R), R about 2e-4.  u = 2^-24.
* z: 32 places of eight chains each.  Chains add up to 2^-17 D / 256 in steps of which
  each is off by u of that: nothing.  Three additions in a place, five of places,
  off by 2^-20 each between 16 and 32: 8 2^-20.
* R, relative: that of z; the exponent, about 23, its rounding and that of log2 e, 2 x
  2^-20 log 2; exponentials and the sums of V of them through chains of fewer than 2^6
  additions: 2^-18.  Altogether 13.4 2^-20, below 2^-16.
* loss, relative: no more than R, as log(1 + R) / R falls.
* dz: a (exp(z - lse) - 1), where lse = z + loss rounded to binary32, off by 2^-20, and
  z is the same number in both; expm1, a's and the loss's roundings: u' = 2^-16 of dz; then a half step of bf16 twice
  (dz, and d_hidden where the target's row holds 1): 2 x 2^-8 of dz."""
import pytest
import torch

V, D = 1003, 4096


def inputs(n, device, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape):
        return torch.rand(*shape, generator=g)
    target = V // 3
    hidden = 2.0 ** -9 * (1 + rand(n, D))
    weight = torch.zeros(V, D)
    weight[target] = 2.0 ** -10 * (0.5 + rand(D))
    chain = torch.arange(D) % 64 == 0                   # where the large term is summed
    hidden[:, chain] = 0
    weight[:, chain] = 0
    hidden[:, 0] = 16
    weight[target, 0] = 1
    hidden[:, 64] = 1 + rand(n)
    weight[:, 64] = 2 * rand(V) - 1
    weight[target, 64] = 0
    hidden, weight = hidden.to(torch.bfloat16), weight.to(torch.bfloat16)
    targets = torch.full((n,), target)
    return [x.to(device) for x in (hidden, weight, targets)]


def exact(hidden, weight, targets):
    """z, the other words' log sum, loss and dz / a, in 64 bits."""
    z = hidden.double() @ weight.double().T
    zy = z.gather(1, targets[:, None])[:, 0]
    rest = z.scatter(1, targets[:, None], -torch.inf).logsumexp(dim=1)
    r = torch.exp(rest - zy)
    return zy, rest, torch.log1p(r), -r / (1 + r)


def bounds(loss, dz):
    return 2.0 ** -16 * loss, 2.0 ** -20 + (2.0 ** -16 + 2.0 ** -7) * dz.abs()


def summed(hidden, weight, targets, lanes):
    """The target's logit by chains of binary32 sums, as the kernels'."""
    x = hidden.float() * weight[targets].float()        # exact
    s = torch.zeros(len(x), lanes, 8)
    for part in x.view(len(x), -1, lanes, 8).unbind(1):
        s = s + part
    while s.shape[2] > 1:
        s = s[:, :, ::2] + s[:, :, 1::2]
    s = s[:, :, 0]
    while s.shape[1] > 1:
        s = s[:, :s.shape[1] // 2] + s[:, s.shape[1] // 2:]
    return s[:, 0]


def cut_off(hidden, weight, targets):
    """The same by steps of 16 exact terms, each sum cut off to binary32."""
    x = (hidden.double() * weight[targets].double()).view(len(hidden), -1, 16).sum(dim=2)
    s = torch.zeros(len(x), dtype=torch.float64)
    for part in x.unbind(1):
        t = s + part
        near = t.float()
        s = torch.where(near.double() > t, torch.nextafter(near, torch.zeros(())), near).double()
    return s.float()


def form(hidden, weight, targets, wrong=None):
    """loss and d_hidden / a at the target's place of 1, in binary32."""
    zy, rest, _, _ = exact(hidden, weight, targets)
    z = (cut_off if wrong == "cut off" else lambda *a: summed(*a, 32))(hidden, weight, targets)
    loss = torch.log1p(torch.exp(rest.float() - z))
    lse = z + loss
    if wrong == "a difference":
        loss = lse - z
    again = z
    if wrong == "another order":
        again = summed(hidden, weight, targets, 8)
    dz = torch.expm1(again - lse)
    if wrong == "cut off in the gradient":
        dz = torch.expm1(cut_off(hidden, weight, targets) - lse)
    return loss, dz.to(torch.bfloat16)


def misses(got, want, bound):
    return int((~((got.double() - want).abs() <= bound)).sum())


def judged(loss, dz, hidden, weight, targets):
    _, _, want, want_dz = exact(hidden, weight, targets)
    assert 1e-4 < float(want.min()) and float(want.max()) < 1e-3
    for_loss, for_dz = bounds(want, want_dz)
    return misses(loss, want, for_loss), misses(dz, want_dz, for_dz)


@pytest.mark.parametrize("seed", range(3))
def test_a_form_without_mistakes_is_inside(seed):
    args = inputs(400, "cpu", seed)
    assert judged(*form(*args), *args) == (0, 0)


@pytest.mark.parametrize("wrong,at", [("cut off", 0), ("a difference", 0), ("another order", 1),
                                      ("cut off in the gradient", 1)])
def test_a_mistake_is_outside(wrong, at):
    args = inputs(400, "cpu")
    assert judged(*form(*args, wrong), *args)[at] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 30, 100, 700])
@pytest.mark.parametrize("weighted", [False, True])
def test_the_kernels_are_inside(n, weighted):
    from optimizer_state_gb300 import z3
    hidden, weight, targets = args = inputs(n, "cuda", n)
    loss, lse = (torch.empty(n, device="cuda") for _ in range(2))
    total = torch.empty(2, device="cuda")
    d_hidden, d_weight = torch.empty_like(hidden), torch.empty_like(weight)
    each = torch.tensor([0.5, 2.0, 0.25], device="cuda").repeat(n)[:n] if weighted else None
    ws = z3.head_workspace(n, D, V)
    z3.z3_xent(hidden, weight, targets, loss, lse, total, ws, weights=each)
    # factors of powers of two: they take no digits
    z3.z3_xent_grad(hidden, weight, targets, lse, None, 4.0, d_hidden, d_weight, ws, weights=each)
    torch.cuda.synchronize()
    # column 0 is the target's alone, where its row holds 1
    dz = d_hidden[:, 0].double() / 4
    if weighted:
        dz /= each
    assert judged(loss, dz, *args) == (0, 0)
    # the same z in the loss as in dz: what lse rounds away is all that is between them
    want = exact(*args)[0] + loss.double()
    assert float((lse.double() - want).abs().max()) <= 9 * 2.0 ** -20
