"""Gradient clipping by the global norm over sharded model state: its cases, and its plain form.

Five operators of ``optimizer_state_gb300.z3`` are run here:

* ``z3_grad_norm``: the L2 norm over many tensors taken as one vector, and the
  factor ``coef`` that brings it down to ``max_norm``;
* ``z3_clip``: those tensors times ``coef``, in place;
* ``z3_reduce_scatter_norm``: the reduce-scatter of N ranks' gradients that
  also leaves the sums of squares of what it stores, for ``z3_grad_norm``;
* ``z3_adam_shard_step_clipped``: the shard Adam update of gradients times
  ``coef``;
* ``z3_model_step_clipped``: a whole training step of many units with all of
  them: gathers, reduce-scatters, one norm over every unit, updates.

Definitions.  With g the concatenation of the tensors, all in binary32 or more,

    norm = sqrt(sum_i g_i^2)
    coef = max_norm / norm where norm > max_norm, else 1; NaN where norm is not finite
    clip:    g_i <- coef * g_i               (nothing is written where coef is NaN)
    reduce:  g = scale * sum_k grads[k] (+ the running sum), cut into the N ranks' slices
    update:  Adam with coef * g as its gradient (nothing is written where coef is NaN)

A rank's shard of a layer is the concatenation of its slices of the layer's
parameters: parameter p of n_p elements is padded with zeros to N * s_p, s_p =
ceil(n_p / N), and rank r keeps positions [r * s_p, (r + 1) * s_p).

``run`` takes the plain form in elementary torch operations where ``own`` is
false, and makes the framework's calls where it is true.
"""
import functools
import math
import random

import torch

own = False

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
STEP = 7              # the Adam step number: the moments hold earlier steps
GRAD_STD = 1e-3
MAX_BYTES = 20e9      # of a drawn case's work

D1024 = dict(kind="model", d=1024, ffn=4096, vocab=0)


def listed():
    return [
        # -- the norm alone: a step that only watches it, or decides on the host
        # the smallest layer of the tests: three parameters, 60 elements; latency
        dict(name="norm_tiny", op="norm", kind="list", sizes="35 13 12", dtype="f32"),
        # many small odd tensors back to back in two buffers: adapters, gains and biases
        dict(name="norm_odd", op="norm", kind="odd", count=700, longest=60001, lengths=3,
             dtype="mixed"),
        # every gradient of the 24-layer model with its embedding, as backward leaves them
        dict(D1024, name="norm_model", op="norm", layers=24, vocab=50257, dtype="bf16"),
        # -- the norm, then the clipping in place: clipping outside the sharded update
        # one layer's bf16 gradients: they fit L2
        dict(D1024, name="clip_layer", op="clip", layers=1, dtype="bf16"),
        dict(name="clip_odd", op="clip", kind="odd", count=300, longest=200003, lengths=5,
             dtype="mixed"),
        # fp32 gradient accumulators of the whole model
        dict(D1024, name="clip_model", op="clip", layers=24, vocab=50257, dtype="f32"),
        # -- the reduce-scatter with the norm
        dict(D1024, name="reduce_layer", op="reduce", layers=1, ranks=8, accumulate=False),
        # three prime-length parameters, whose chunks need shifted windows; many
        # ranks; the last micro-batch, added to the running sums
        dict(name="reduce_primes", op="reduce", kind="list", sizes="8388617 4194319 1048583",
             ranks=64, accumulate=True),
        # -- the clipped update
        dict(D1024, name="adam_layer", op="adam", layers=1, ranks=8),
        # one flattened prime-length parameter of the sweep
        dict(name="adam_sweep", op="adam", kind="list", sizes="67108879", ranks=2),
        # -- the whole clipped step: one layer, and the 24-layer model with its embedding
        dict(D1024, name="step_layer", op="step", layers=1, ranks=8),
        dict(D1024, name="step_model", op="step", layers=24, vocab=50257, ranks=16),
    ]


def _between(rng, lo, hi):
    """A whole number, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "clip", "reduce", "adam", "step"])
        kind = rng.choice(["model", "odd", "list"])
        if op == "step":
            kind = rng.choice(["model", "odd"])
        case = dict(op=op, kind=kind)
        if kind == "model":
            case |= dict(d=8 * _between(rng, 4, 128), layers=_between(rng, 1, 24),
                         vocab=rng.choice([0, _between(rng, 100, 50257)]))
            case["ffn"] = case["d"] * rng.choice([2, 4]) + rng.choice([0, 0, 24])
        elif kind == "odd":
            case |= dict(count=_between(rng, 1, 1500 if op in ("norm", "clip") else 90),
                         longest=_between(rng, 1, 400000), lengths=rng.randrange(1000))
        else:
            case |= dict(sizes=" ".join(str(_between(rng, 1, 150_000_000))
                                        for _ in range(rng.randint(1, 3))))
        if op in ("norm", "clip"):
            case["dtype"] = rng.choice(["bf16", "f32", "mixed"])
        else:
            case["ranks"] = _between(rng, 1, 64)
        if op == "reduce":
            case["accumulate"] = rng.random() < 0.5
        if work(case)["bytes"] <= MAX_BYTES:
            return case


def units_of(case):
    """The units' parameter lengths: a list of lists."""
    if case["kind"] == "model":
        d, f = case["d"], case["ffn"]
        layer = [3 * d * d, d * d, f * d, d * f, d, d]
        return ([[case["vocab"] * d]] if case["vocab"] else []) + [layer] * case["layers"]
    if case["kind"] == "odd":
        r = random.Random(case["lengths"])
        lengths = [int(case["longest"] ** r.random()) for _ in range(case["count"])]
        return [lengths[i:i + 7] for i in range(0, len(lengths), 7)]
    return [[int(x) for x in case["sizes"].split()]]


def work(case):
    units = units_of(case)
    n = sum(map(sum, units))
    if case["op"] in ("norm", "clip"):
        size = sum(x * (2 if case["dtype"] == "bf16" or case["dtype"] == "mixed" and i % 2 else 4)
                   for i, x in enumerate(y for u in units for y in u))
        return {"bytes": size * (1 if case["op"] == "norm" else 2),
                "flops": n * (2 if case["op"] == "norm" else 3)}
    ranks = case["ranks"]
    if case["op"] == "reduce":
        return {"bytes": n * (2 * ranks + (8 if case["accumulate"] else 4)),
                "flops": n * (ranks + 3)}
    if case["op"] == "adam":
        return {"bytes": n * 30, "flops": n * 18}
    # gradients, the gathered copy, master, m and v read and written, shards written
    return {"bytes": n * (2 * ranks + 4 + 26), "flops": n * (ranks + 20)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(n, std, dtype, gen):
    """N(0, std) in `dtype`, drawn on the device in pieces."""
    out = torch.empty(n, dtype=dtype, device="cuda")
    for at in range(0, n, 1 << 28):
        out[at:at + (1 << 28)].normal_(0.0, std, generator=gen)
    return out


def _pitch(n):
    return -(-n // 8) * 8


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    units = units_of(case)
    state = dict(case=case, units=units)
    if case["op"] in ("norm", "clip"):
        # the tensors lie back to back in one buffer for each type
        sizes = [x for u in units for x in u]
        kinds = [torch.bfloat16 if case["dtype"] == "bf16" or case["dtype"] == "mixed" and i % 2
                 else torch.float32 for i in range(len(sizes))]
        buffers, tensors = {}, []
        for dt in dict.fromkeys(kinds):
            buffers[dt] = _normal(sum(x for x, k in zip(sizes, kinds) if k == dt), GRAD_STD, dt,
                                  gen)
        at = dict.fromkeys(buffers, 0)
        for x, k in zip(sizes, kinds):
            tensors.append(buffers[k][at[k]:at[k] + x])
            at[k] += x
        state |= dict(buffers=list(buffers.values()), tensors=tensors,
                      max_norm=0.37 * GRAD_STD * math.sqrt(sum(sizes)))
    else:
        ranks = case["ranks"]
        numel = [x for u in units for x in u]
        if case["op"] == "step":
            groups = units
        else:
            groups = units = state["units"] = [numel]
        state["max_norm"] = 0.37 * GRAD_STD * math.sqrt(sum(numel) / ranks)
        if case["op"] in ("reduce", "step"):
            state["grads"] = []
            for u in groups:
                g = _normal(ranks * _pitch(sum(u)), GRAD_STD, torch.bfloat16, gen)
                state["grads"].append(g.view(ranks, _pitch(sum(u))))
        # every unit's [N][S] buffers are pieces of one buffer, each on a 16-byte boundary
        padded = [ranks * sum(-(-x // ranks) for x in u) for u in groups]
        state["padded"] = padded
        starts = [sum(map(_pitch, padded[:i])) for i in range(len(groups))]
        state["spans"] = [(a, a + n) for a, n in zip(starts, padded)]
        total = sum(map(_pitch, padded))
        # 1 where a position is an element, 0 in the pads
        real = torch.zeros(total, dtype=torch.bool, device="cuda")
        for (a, b), u in zip(state["spans"], groups):
            real[a:b] = _to_shards([torch.ones(x, dtype=torch.bool, device="cuda") for x in u],
                                   ranks)

        def values(std):
            return _normal(total, std, torch.float32, gen).mul_(real)
        if case["op"] == "reduce" and case["accumulate"]:
            state["grad_shards"] = values(GRAD_STD / math.sqrt(ranks))
        elif case["op"] in ("reduce", "step"):
            state["grad_shards"] = torch.zeros(total, dtype=torch.float32, device="cuda")
        else:
            state["grad_shards"] = values(GRAD_STD)
            # what z3_grad_norm left: the norm over all units, and its factor
            state["clip"] = torch.tensor([GRAD_STD * 1e5, 0.43], dtype=torch.float32,
                                         device="cuda")
        if case["op"] in ("adam", "step"):
            state["master"] = values(0.02)
            state["m"] = values(0.3 * GRAD_STD)
            state["v"] = values(GRAD_STD).square_()
            state["shards"] = state["master"].to(torch.bfloat16)
        if case["op"] == "step":
            state["full"] = torch.empty(max(map(sum, groups)), dtype=torch.bfloat16,
                                        device="cuda")
        del real
    if own:
        _handles(state)
    return state


def _handles(state):
    """What a program of the framework keeps between steps: layouts, the
    tensor list, the norm's workspace and outputs."""
    from optimizer_state_gb300 import z3
    case = state["case"]
    state["z3"] = z3
    state["workspace"] = z3.grad_norm_workspace()
    if "clip" not in state:
        state["clip"] = torch.zeros(2, dtype=torch.float32, device="cuda")
    if case["op"] in ("norm", "clip"):
        state["list"] = z3.TensorList(state["tensors"])
        return
    state["layouts"] = [z3.Layout(u, case["ranks"]) for u in state["units"]]

    def parts(name):
        return [state[name][a:b] for a, b in state["spans"]]
    if case["op"] in ("reduce", "step"):
        state["sumsq"] = [torch.zeros(L.sumsq_len, dtype=torch.float64, device="cuda")
                          for L in state["layouts"]]
        state["list"] = z3.TensorList([], sumsq=state["sumsq"])
    if case["op"] == "step":
        scale = 1.0 / case["ranks"]
        state["args"] = list(zip(state["layouts"], parts("shards"), parts("master"), parts("m"),
                                 parts("v"), state["grads"],
                                 [g.shape[1] for g in state["grads"]],
                                 [scale] * len(state["layouts"])))
        state["clip_args"] = list(zip(parts("grad_shards"), state["sumsq"]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    out = {"norm": _run_norm, "clip": _run_clip, "reduce": _run_reduce, "adam": _run_adam,
           "step": _run_step}[op](state)
    return out


def _run_norm(state):
    if own:
        state["z3"].z3_grad_norm(state["list"], state["max_norm"], state["clip"],
                                 state["workspace"])
        return {"clip": state["clip"]}
    return {"clip": _plain_norm(state["tensors"], state["max_norm"])}


def _run_clip(state):
    # the bound of a program that lowers it a little each step: the gradients
    # of a second pass, clipped by the first, are above it again
    max_norm, state["max_norm"] = state["max_norm"], state["max_norm"] * 0.9999
    if own:
        z3 = state["z3"]
        z3.z3_grad_norm(state["list"], max_norm, state["clip"], state["workspace"])
        z3.z3_clip(state["list"], state["clip"])
        return {"clip": state["clip"], "buffers": state["buffers"]}
    clip = _plain_norm(state["tensors"], max_norm)
    coef = torch.where(clip[1].isnan(), 1.0, clip[1])
    _ = [t.copy_(t.float() * coef) for t in state["tensors"]]
    return {"clip": clip, "buffers": state["buffers"]}


def _run_reduce(state):
    case, grads, out = state["case"], state["grads"][0], state["grad_shards"]
    scale = 1.0 / case["ranks"]
    if own:
        z3 = state["z3"]
        z3.z3_reduce_scatter_norm(state["layouts"][0], grads, grads.shape[1], out, scale,
                                  state["sumsq"][0], accumulate=case["accumulate"])
        z3.z3_grad_norm(state["list"], state["max_norm"], state["clip"], state["workspace"])
        return {"clip": state["clip"], "grad_shards": out}
    _plain_reduce(grads, state["units"][0], scale, out[:state["padded"][0]], case["accumulate"])
    return {"clip": _plain_norm([out], state["max_norm"]), "grad_shards": out}


def _run_adam(state):
    names = ("master", "m", "v", "grad_shards", "shards")
    if own:
        state["z3"].z3_adam_shard_step_clipped(state["layouts"][0], *[state[x] for x in names],
                                               HP, STEP, state["clip"])
    else:
        _plain_adam(*[state[x] for x in names], state["clip"])
    return {x: state[x] for x in ("master", "m", "v", "shards")}


def _run_step(state):
    if own:
        state["z3"].z3_model_step_clipped(state["args"], state["clip_args"], [state["full"]], HP,
                                          STEP, state["max_norm"], state["clip"],
                                          state["workspace"])
        return {x: state[x] for x in ("clip", "grad_shards", "master", "m", "v", "shards")}
    ranks = state["case"]["ranks"]
    everything = list(zip(state["units"], state["spans"]))
    _ = [_plain_gather(state["shards"][a:b], u, ranks, state["full"])
         for u, (a, b) in everything]
    _ = [(_plain_gather(state["shards"][a:b], u, ranks, state["full"]),
          _plain_reduce(g, u, 1.0 / ranks, state["grad_shards"][a:b], False))
         for (u, (a, b)), g in reversed(list(zip(everything, state["grads"])))]
    clip = _plain_norm([state["grad_shards"][a:b] for _, (a, b) in everything],
                       state["max_norm"])
    _ = [_plain_adam(*[state[x][a:b] for x in ("master", "m", "v", "grad_shards", "shards")],
                     clip) for _, (a, b) in everything]
    return {"clip": clip, **{x: state[x] for x in ("grad_shards", "master", "m", "v", "shards")}}


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _plain_norm(tensors, max_norm):
    """[norm, coef] in 32 bits."""
    norm = torch.stack([t.float().square().sum() for t in tensors]).sum().sqrt()
    coef = torch.where(norm > max_norm, max_norm / norm, 1.0)
    return torch.stack([norm, torch.where(norm.isfinite(), coef, math.nan)])


def _to_shards(parts, ranks):
    """The parameters' flat values as the N ranks' shards, one after the other."""
    cut = [torch.nn.functional.pad(x, (0, -x.numel() % ranks)).view(ranks, -1) for x in parts]
    return torch.cat(cut, dim=1).view(-1)


def _plain_reduce(grads, numel, scale, out, accumulate):
    full = functools.reduce(lambda s, g: s.add_(g.float()), grads[1:], grads[0].float())
    got = _to_shards((full[:sum(numel)] * scale).split(numel), len(grads))
    out.copy_(out + got if accumulate else got)


def _plain_gather(shards, numel, ranks, full):
    s = [-(-x // ranks) for x in numel]
    parts = shards.view(ranks, -1).split(s, dim=1)
    full[:sum(numel)] = torch.cat([p.reshape(-1)[:x] for p, x in zip(parts, numel)])


def _plain_adam(master, m, v, grad, shards, clip):
    b1, b2 = HP["beta1"], HP["beta2"]
    skip = clip[1].isnan()
    g = grad * clip[1]
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * (g * g)
    u = (m1 * (1 / (1 - b1 ** STEP))) / ((v1 * (1 / (1 - b2 ** STEP))).sqrt() + HP["eps"])
    p = (master - HP["lr"] * HP["weight_decay"] * master) - HP["lr"] * u
    _ = [x.copy_(torch.where(skip, x, y)) for x, y in ((master, p), (m, m1), (v, v1))]
    shards.copy_(torch.where(skip, shards, p.to(torch.bfloat16)))


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain form
# ---------------------------------------------------------------------------

def _exact_clip(squares, max_norm):
    norm = math.sqrt(squares)
    coef = math.nan if not math.isfinite(norm) else max_norm / norm if norm > max_norm else 1.0
    return torch.tensor([norm, coef], dtype=torch.float64), coef


def _exact_shards(grads, numel, scale):
    """The reduced gradient in the shard order, by index: position (r, j) of
    parameter p is its element r * s_p + j, or pad."""
    ranks = grads.shape[0]
    total = torch.zeros(grads.shape[1], dtype=torch.float64, device=grads.device)
    for k in range(ranks):
        total += grads[k]
    total *= scale
    widths = [-(-x // ranks) for x in numel]
    out = torch.zeros(ranks, sum(widths), dtype=torch.float64, device=grads.device)
    first, column = 0, 0
    for x, s in zip(numel, widths):
        for r in range(ranks):
            here = max(0, min(s, x - r * s))
            out[r, column:column + here] = total[first + r * s:first + r * s + here]
        first, column = first + x, column + s
    return out.view(-1)


def _exact_adam(p, m, v, g, t):
    """Kingma & Ba, Algorithm 1, with decoupled weight decay, in place of p, m, v."""
    m.mul_(HP["beta1"]).add_(g, alpha=1 - HP["beta1"])
    v.mul_(HP["beta2"]).addcmul_(g, g, value=1 - HP["beta2"])
    p.mul_(1 - HP["lr"] * HP["weight_decay"])
    root = (v / (1 - HP["beta2"] ** t)).sqrt_().add_(HP["eps"])
    p.sub_((m / (1 - HP["beta1"] ** t)).div_(root), alpha=HP["lr"])


def exact(case, seed):
    global own
    kept, own = own, False          # the inputs alone, without the framework's handles
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op in ("norm", "clip"):
        squares = sum(float(b.double().square_().sum()) for b in state["buffers"])
        clip, coef = _exact_clip(squares, state["max_norm"])
        if op == "norm":
            return {"clip": clip}
        return {"clip": clip, "buffers": [b.double().mul_(coef) for b in state["buffers"]]}
    g, coef = state["grad_shards"].double(), None
    if op in ("reduce", "step"):
        squares = 0.0
        for u, (a, b), x in zip(state["units"], state["spans"], state["grads"]):
            g[a:b] += _exact_shards(x, u, 1.0 / case["ranks"])
            squares += float(g[a:b].square().sum())
        clip, coef = _exact_clip(squares, state["max_norm"])
        if op == "reduce":
            return {"clip": clip, "grad_shards": g}
        del state["grads"]
    else:
        coef = float(state["clip"][1].double())
    out = {x: state[x].double() for x in ("master", "m", "v")}
    _exact_adam(out["master"], out["m"], out["v"], g * coef, STEP)
    out["shards"] = out["master"]
    if op == "step":
        out |= {"clip": clip, "grad_shards": g}
    return out
