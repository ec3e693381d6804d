"""Losses over a large vocabulary, without keeping its logits: their cases, and their plain form.

Four operators of ``optimizer_state_gb300.z3`` are run here, on the hidden
states [tokens, dim] that a model's last layer leaves and on the head's weight
[vocab, dim], the gathered bf16 copy of the head's (or a tied embedding's) unit:

* ``z3_xent``: softmax cross entropy against one target a token;
* ``z3_xent_grad``: its gradient for the hidden states and for the weight, the
  latter being what a rank hands to the reduce-scatter;
* ``z3_distill``: the divergence from a teacher whose top logits are given;
* ``z3_distill_grad``: its gradient.

Definitions.  With z = hidden weight^T, y the targets, tau the temperature,

    xent:     lse_t = log sum_j exp z_tj,          loss_t = lse_t - z_ty
    distill:  q_t = softmax(teacher_t / tau) over the k logits given
              lse_t = log sum_j exp(z_tj / tau)
              loss_t = tau^2 sum_k q_tk (log q_tk - z_t,index(k) / tau + lse_t)
    total = [sum_t w_t loss_t, sum_t w_t]

over the tokens that count: a negative target leaves a token out, a negative
index leaves out an entry of a token's list, and a token without entries is
left out.  w is 1, or given.  A token left out has loss and lse 0.  The gradient
is that of scale * total[0] / total[1]:

    dz_tj = (scale w_t / total[1]) (p_tj - [j = y_t]),              p = exp(z - lse)
    dz_tj = (scale w_t / total[1]) tau (p_tj - sum_{k: index = j} q_tk),  p = exp(z / tau - lse)
    d_hidden = dz weight,   d_weight = dz^T hidden

``run`` takes the plain form in elementary torch operations where ``own`` is
false, and makes the framework's calls where it is true.
"""
import math

import torch

own = False

SCALE = 0.5           # of the gradient: one of two micro-batches
MAX_FLOPS = 6.0 * 2048 * 131072 * 4096

# the 24-layer workload's embedding, tied as its head
MODEL = dict(vocab=50257, dim=1024, ignored=0.0, weighted=False)


def listed():
    return [
        # -- the loss alone: evaluation, scoring
        # one token's score against the whole vocabulary: latency, one read of the weight
        dict(MODEL, name="xent_one", op="xent", tokens=1),
        # eight sequences of 1024
        dict(MODEL, name="xent_model", op="xent", tokens=8192),
        # odd sizes, padded rows, tokens weighted
        dict(name="xent_odd", op="xent", tokens=1999, vocab=10007, dim=520, ignored=0.3,
             weighted=True),
        # a 7B-style model's width with a large vocabulary
        dict(name="xent_wide", op="xent", tokens=4096, vocab=131072, dim=4096, ignored=0.0,
             weighted=False),
        # -- a training step of the head: the loss, then both gradients
        # a few tokens: every pass over the weight counts
        dict(MODEL, name="xent_train_few", op="xent_train", tokens=16),
        dict(MODEL, name="xent_train_model", op="xent_train", tokens=8192, ignored=0.1),
        dict(name="xent_train_odd", op="xent_train", tokens=3001, vocab=32003, dim=1032,
             ignored=0.3, weighted=True),
        dict(name="xent_train_wide", op="xent_train", tokens=2048, vocab=131072, dim=4096,
             ignored=0.0, weighted=False),
        # -- distillation: the loss alone
        dict(MODEL, name="distill_model", op="distill", tokens=4096, k=64, teacher="bf16",
             temperature=2.0),
        dict(name="distill_odd", op="distill", tokens=777, vocab=10007, dim=520, k=19,
             teacher="f32", temperature=1.0, ignored=0.3, weighted=True),
        # -- and a training step
        dict(MODEL, name="distill_train_model", op="distill_train", tokens=4096, k=64,
             teacher="bf16", temperature=2.0, ignored=0.1),
        dict(name="distill_train_odd", op="distill_train", tokens=501, vocab=32003, dim=1032,
             k=200, teacher="f32", temperature=1.5, ignored=0.3, weighted=True),
    ]


def _between(rng, lo, hi):
    """A whole number, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = dict(op=rng.choice(["xent", "xent_train", "distill", "distill_train"]),
                    tokens=_between(rng, 1, 16384), vocab=_between(rng, 300, 131072),
                    dim=8 * _between(rng, 8, 512), ignored=rng.choice([0.0, 0.1, 0.5]),
                    weighted=rng.random() < 0.3)
        if case["op"].startswith("distill"):
            case |= dict(k=_between(rng, 1, 256), teacher=rng.choice(["bf16", "f32"]),
                         temperature=rng.choice([1.0, 1.5, 2.0, 4.0]))
        if work(case)["flops"] <= MAX_FLOPS:
            return case


def work(case):
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    train = case["op"].endswith("_train")
    size = 2 * (n + v) * d * (2 if train else 1) + 8 * n + (4 * n if case["weighted"] else 0)
    if case["op"].startswith("distill"):
        size += n * case["k"] * (8 + (2 if case["teacher"] == "bf16" else 4))
    else:
        size += 8 * n
    return {"bytes": size, "flops": (6 if train else 2) * n * v * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, v, d = case["tokens"], case["vocab"], case["dim"]

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    std = 0.02
    weight = torch.empty(v, d, dtype=torch.bfloat16, device="cuda").normal_(0.0, std,
                                                                           generator=gen)
    # words as text has them: a few often, most seldom
    words = (v ** uniform(n)).long().sub_(1).clamp_(0, v - 1)
    # normalised hidden states that know their word: its logit is up to 14 higher
    hidden = torch.empty(n, d, device="cuda").normal_(0.0, 1.0, generator=gen)
    hidden += (14 * uniform(n, 1) / (std * std * d)) * weight[words].float()
    hidden = hidden.to(torch.bfloat16)
    left_out = uniform(n) < case["ignored"]
    state = dict(case=case, hidden=hidden, weight=weight, weights=None)
    if case["weighted"]:
        state["weights"] = 0.25 + uniform(n)
    if case["op"].startswith("distill"):
        k = case["k"]
        # the word, then others spread over the vocabulary: all distinct
        step = 1 + (uniform(n, 1) * ((v - 1) // k)).long()
        index = (words[:, None] + step * torch.arange(k, device="cuda")) % v
        teacher, _ = torch.empty(n, k, device="cuda").normal_(0.0, 2.0, generator=gen).sort(
            dim=1, descending=True)
        teacher[:, 0] += 6 * uniform(n)
        # lists of different lengths, some of them empty
        kept = 1 + (uniform(n, 1) * k).long()
        index.masked_fill_(torch.arange(k, device="cuda") >= kept, -1)
        index.masked_fill_(left_out[:, None], -1)
        state |= dict(index=index, temperature=case["temperature"], teacher=teacher.to(
            torch.bfloat16 if case["teacher"] == "bf16" else torch.float32))
    else:
        state["targets"] = words.masked_fill_(left_out, -100)
    # what the step writes to
    state |= dict(loss=torch.empty(n, device="cuda"), lse=torch.empty(n, device="cuda"),
                  total=torch.empty(2, device="cuda"))
    if case["op"].endswith("_train"):
        state |= dict(d_hidden=torch.empty_like(hidden), d_weight=torch.empty_like(weight))
    if own:
        from optimizer_state_gb300 import z3
        state["z3"] = z3
        state["workspace"] = z3.head_workspace(n, d, v, k=case.get("k", 0),
                                               grads=case["op"].endswith("_train"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"xent": _run_xent, "xent_train": _run_xent, "distill": _run_distill,
            "distill_train": _run_distill}[state["case"]["op"]](state)


def _outputs(state):
    return {x: state[x] for x in ("loss", "lse", "total", "d_hidden", "d_weight") if x in state}


def _run_xent(state):
    hidden, weight, targets = state["hidden"], state["weight"], state["targets"]
    if own:
        z3, ws = state["z3"], state["workspace"]
        z3.z3_xent(hidden, weight, targets, state["loss"], state["lse"], state["total"], ws,
                   weights=state["weights"])
        if "d_hidden" in state:
            z3.z3_xent_grad(hidden, weight, targets, state["lse"], state["total"], SCALE,
                            state["d_hidden"], state["d_weight"], ws, weights=state["weights"])
        return _outputs(state)
    z, lse = _plain_softmax(hidden, weight, 1.0)
    counts = targets >= 0
    at = targets.clamp(min=0)[:, None]
    loss = lse - z.gather(1, at)[:, 0]
    a = _plain_total(state, loss, lse, counts)
    if "d_hidden" in state:
        dz = z.sub_(lse[:, None]).exp_()
        dz.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=dz.dtype))
        _plain_grads(state, dz, a, counts)
    return _outputs(state)


def _run_distill(state):
    hidden, weight, index = state["hidden"], state["weight"], state["index"]
    tau = state["temperature"]
    if own:
        z3, ws = state["z3"], state["workspace"]
        z3.z3_distill(hidden, weight, state["teacher"], index, tau, state["loss"], state["lse"],
                      state["total"], ws, weights=state["weights"])
        if "d_hidden" in state:
            z3.z3_distill_grad(hidden, weight, state["teacher"], index, tau, state["lse"],
                               state["total"], SCALE, state["d_hidden"], state["d_weight"], ws,
                               weights=state["weights"])
        return _outputs(state)
    z, lse = _plain_softmax(hidden, weight, 1.0 / tau)
    there = index >= 0
    counts = there.any(dim=1)
    t = (state["teacher"].float() / tau).masked_fill(~there, -math.inf)
    t = t - t.amax(dim=1, keepdim=True).masked_fill(~counts[:, None], 0.0)
    e = t.exp()
    norm = e.sum(dim=1, keepdim=True).masked_fill(~counts[:, None], 1.0)
    q = e / norm
    at = index.clamp(min=0)
    log_ratio = (t - norm.log()).masked_fill(~there, 0.0) - z.gather(1, at) + lse[:, None]
    loss = tau * tau * (q * log_ratio).sum(dim=1)
    a = _plain_total(state, loss, lse, counts)
    if "d_hidden" in state:
        dz = z.sub_(lse[:, None]).exp_()
        dz.scatter_add_(1, at, -q)
        _plain_grads(state, dz, a * tau, counts)
    return _outputs(state)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _plain_softmax(hidden, weight, beta):
    """beta * logits and the logarithm of their exponentials' sums, in 32 bits."""
    z = (hidden.float() @ weight.float().t()).mul_(beta)
    top = z.amax(dim=1)
    return z, top + (z - top[:, None]).exp_().sum(dim=1).log()


def _plain_total(state, loss, lse, counts):
    """Writes loss, lse and total, and returns each token's factor."""
    w = counts.float() if state["weights"] is None else state["weights"] * counts
    state["loss"].copy_(torch.where(counts, loss, 0.0))
    state["lse"].copy_(torch.where(counts, lse, 0.0))
    state["total"].copy_(torch.stack([(w * state["loss"]).sum(), w.sum()]))
    total = state["total"][1]
    return torch.where(total != 0, SCALE * w / total, 0.0)


def _plain_grads(state, dz, a, counts):
    dz = torch.where(counts[:, None], dz * a[:, None], 0.0)
    state["d_hidden"].copy_(dz @ state["weight"].float())
    state["d_weight"].copy_(dz.t() @ state["hidden"].float())


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain form
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False          # the inputs alone, without the framework's workspace
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    n, train = case["tokens"], case["op"].endswith("_train")
    w64 = state["weight"].double()
    each = (torch.ones(n, dtype=torch.float64, device="cuda") if state["weights"] is None
            else state["weights"].double())
    tau = case.get("temperature", 1.0)
    if case["op"].startswith("distill"):
        counts = (state["index"] >= 0).sum(dim=1) > 0
    else:
        counts = ~(state["targets"] < 0)
    each = each * counts
    mass = float(each.sum())
    out = dict(loss=torch.zeros(n, dtype=torch.float64, device="cuda"),
               lse=torch.zeros(n, dtype=torch.float64, device="cuda"))
    if train:
        out |= dict(d_hidden=torch.zeros(n, case["dim"], dtype=torch.float64, device="cuda"),
                    d_weight=torch.zeros_like(w64))
    for first in range(0, n, 512):                       # some tokens at a time
        rows = slice(first, min(n, first + 512))
        h64 = state["hidden"][rows].double()
        logp = torch.nn.functional.log_softmax(torch.mm(h64, w64.T) / tau, dim=-1)
        z0 = (h64 * w64[0]).sum(dim=1) / tau              # the first word's logit gives lse
        goal = torch.zeros_like(logp)                     # the distribution aimed at
        if case["op"].startswith("distill"):
            idx, given = state["index"][rows], state["teacher"][rows].double() / tau
            q = torch.softmax(given.masked_fill(idx < 0, -1e300), dim=-1)
            q = torch.where(idx < 0, 0.0, q)
            goal.scatter_add_(1, idx.clamp(min=0), q)
            entropy = torch.special.entr(q).sum(dim=1)
        else:
            y = state["targets"][rows]
            goal[torch.arange(len(y), device="cuda"), y.clamp(min=0)] = 1.0
            entropy = 0.0
        here = counts[rows]
        loss = tau * tau * (-(goal * logp).sum(dim=1) - entropy)
        out["loss"][rows] = torch.where(here, loss, 0.0)
        out["lse"][rows] = torch.where(here, z0 - logp[:, 0], 0.0)
        if train and mass:
            dz = (logp.exp() - goal) * (SCALE * tau / mass * each[rows])[:, None]
            dz[~here] = 0.0
            out["d_hidden"][rows] = torch.mm(dz, w64)
            out["d_weight"] += torch.mm(dz.T, h64)
    out["total"] = torch.stack([(each * out["loss"]).sum(), each.sum()])
    names = ("loss", "lse", "total", "d_hidden", "d_weight")
    return {x: out[x] for x in names if x in out}
