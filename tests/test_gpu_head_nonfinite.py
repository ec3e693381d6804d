"""Losses over a vocabulary where a logit that the loss names is not finite: the
token's loss and lse are NaN, and its gradients with them; no other token's
loss is."""
import pytest
import torch

from head_reference import outside, reference
from optimizer_state_gb300 import z3

pytestmark = pytest.mark.gpu

TOKEN = 2                 # the one that is spoilt
INF = float("inf")


class Call:
    """Tokens of which one alone asks for the word in the middle."""

    def __init__(self, n, v, k, d=72, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.rand(*shape, device="cuda", generator=g)
        self.n, self.v, self.d, self.k = n, v, d, k
        self.word = v // 2
        self.weight = (torch.randn(v, d, device="cuda", generator=g) * d ** -0.5).to(torch.bfloat16)
        self.hidden = torch.randn(n, d, device="cuda", generator=g).to(torch.bfloat16)
        self.tau = 2.0 if k else 1.0
        self.targets = self.index = self.teacher = None
        shape = (n, k) if k else (n,)
        words = (rand(*shape) * (v - 1)).long().clamp(max=max(v - 2, 0))
        words += (words >= self.word).long() * (v > 1)         # any but that one
        if k:
            words[TOKEN, k - 1] = self.word
            self.index = words
            self.teacher = torch.randn(n, k, device="cuda", generator=g)
        else:
            words[TOKEN] = self.word
            self.targets = words

    def run(self):
        f32, dev = torch.float32, "cuda"
        t = dict(loss=torch.empty(self.n, dtype=f32, device=dev),
                 lse=torch.empty(self.n, dtype=f32, device=dev),
                 total=torch.empty(2, dtype=f32, device=dev),
                 d_hidden=torch.empty_like(self.hidden), d_weight=torch.empty_like(self.weight))
        ws = z3.head_workspace(self.n, self.d, self.v, k=self.k)
        kind = (self.teacher, self.index, self.tau) if self.k else (self.targets,)
        forward, grad = ((z3.z3_distill, z3.z3_distill_grad) if self.k
                         else (z3.z3_xent, z3.z3_xent_grad))
        forward(self.hidden, self.weight, *kind, t["loss"], t["lse"], t["total"], ws)
        grad(self.hidden, self.weight, *kind, t["lse"], None, 1.0, t["d_hidden"], t["d_weight"],
             ws)
        torch.cuda.synchronize()
        return t

    def others(self):
        return torch.arange(self.n, device="cuda") != TOKEN

    def reference(self, without_word):
        """Of the other tokens, with the whole vocabulary or without the one word."""
        rows = self.others()
        w, words = self.weight, [None if x is None else x[rows] for x in (self.targets, self.index)]
        if without_word:
            w = torch.cat([w[:self.word], w[self.word + 1:]])
            words = [None if x is None else x - (x > self.word).long() for x in words]
        return reference(self.hidden[rows], w, words[0], words[1],
                         None if self.teacher is None else self.teacher[rows], self.tau,
                         mean=False)


def check(c, t, without_word, names):
    rows = c.others()
    for x in ("loss", "lse"):
        assert bool(t[x][TOKEN].isnan()), x
    assert bool(t["total"][0].isnan()) and float(t["total"][1]) == c.n
    assert outside({x: t[x][rows] for x in names}, c.reference(without_word)) == {}
    assert bool(t["d_hidden"][TOKEN].isnan().all()) and bool(t["d_weight"].isnan().all())


SIZES = [(3, 300), (40, 700), (200, 1003), (600, 2500)]


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("k", [0, 4, 70])
@pytest.mark.parametrize("value", [INF, -INF])
def test_an_infinity_in_the_words_weight(n, v, k, value):
    """The word's logit is the token's only one that is not finite.  The others'
    is -Inf, a probability of 0."""
    c = Call(n, v, k)
    c.weight[c.word, 0] = value
    c.hidden[:, 0] = -1.0 if value > 0 else 1.0
    c.hidden[TOKEN, 0] = 1.0
    check(c, c.run(), True, ("loss", "lse"))


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("k", [0, 4, 70])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_logit_beyond_binary32(n, v, k, sign):
    """Finite values whose product is not: the other tokens keep their gradients."""
    c = Call(n, v, k)
    c.weight[:, 0] = 0.0
    c.hidden[:, 0] = 0.0
    c.weight[c.word, 0] = sign * 3e38
    c.hidden[TOKEN, 0] = 3e38
    rows = c.others()
    t = c.run()
    check(c, t, False, ("loss", "lse"))
    ref = c.reference(False)
    # column 0 of the word's weight is 3e38 itself: its share of d_hidden is another test's
    value, bound = ref["d_hidden"]
    assert outside(dict(d_hidden=t["d_hidden"][rows][:, 1:]),
                   dict(d_hidden=(value[:, 1:], bound[:, 1:]))) == {}


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("k", [0, 2])
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
def test_a_vocabulary_of_one(n, k, value):
    c = Call(n, 1, k)
    c.hidden[TOKEN, 3] = value
    t = c.run()
    rows = c.others()
    assert bool(t["loss"][TOKEN].isnan()) and bool(t["lse"][TOKEN].isnan())
    assert bool(t["d_hidden"][TOKEN].isnan().all())
    assert outside({x: t[x][rows] for x in ("loss", "lse")}, c.reference(False)) == {}


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("k", [0, 4])
def test_all_logits_minus_infinity(n, k):
    c = Call(n, 300, k)
    c.weight[:, 0] = 1.0
    c.hidden[TOKEN, 0] = -INF
    t = c.run()
    check(c, t, False, ("loss", "lse"))


@pytest.mark.parametrize("n", [3, 200])
def test_a_listed_word_without_a_share(n):
    """An entry left out, or one whose share is below binary32, is not named."""
    c = Call(n, 300, 4)
    c.weight[c.word, 0] = -INF
    c.hidden[:, 0] = 1.0
    c.teacher[TOKEN, 3] = -INF
    t = c.run()
    assert bool(t["loss"].isfinite().all())
    c.teacher[TOKEN, 3] = -1e30
    # the same shares, added up in another order: their sum moves by 3 additions'
    # roundings, 2^-22 of it, and so do terms of at most 32, times tau^2 = 4
    assert float((c.run()["loss"] - t["loss"]).abs().max()) <= 4 * 32 * 2.0 ** -20
