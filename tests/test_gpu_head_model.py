"""A model's head on its units: the loss of every logical rank over the gathered
embedding, its gradient in the ranks' rows, and the step that follows."""
import pytest
import torch

from head_reference import outside, reference
from optimizer_state_gb300 import inputs as I

pytestmark = pytest.mark.gpu

N, T, V, D = 4, 70, 1003, 64
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)


@pytest.fixture(scope="module")
def sch():
    from optimizer_state_gb300 import build, schedule, z3
    build.build()
    z3.load()
    return schedule


def units(sch, resident=False, lead=()):
    """An embedding, behind parameters `lead` of its unit, and two layers."""
    dev = torch.device("cuda")
    gen = I.make_generator(3, dev)
    emb = I.Workload("embed", lead + ((V, D),), N, 0.02, 1e-3, resident=resident)
    layer = I.Workload("layer", I.transformer_layer_shapes(D, 128, gated=False), N, 0.02, 1e-3)
    return [sch.Unit(w, dev, gen) for w in (emb, layer, layer)]


def batch(k=0):
    g = torch.Generator(device="cuda").manual_seed(5)
    hidden = torch.randn(N, T, D, device="cuda", generator=g).to(torch.bfloat16)
    if k == 0:
        y = torch.randint(0, V, (N, T), device="cuda", generator=g)
        y[torch.rand(N, T, device="cuda", generator=g) < 0.3] = -100
        y[1] = -1                                    # a rank without tokens
        return hidden, dict(targets=y)
    return hidden, dict(teacher=torch.randn(N, T, k, device="cuda", generator=g),
                        index=torch.randint(-1, V, (N, T, k), device="cuda", generator=g),
                        temperature=2.0)


def check(sch, model, head, hidden, given, param=0):
    u = model.units[0]
    full = torch.empty(u.L.psi, dtype=torch.bfloat16, device="cuda")
    from optimizer_state_gb300 import z3
    z3.z3_allgather(u.L, u.shards, full)
    first = u.L.full_off[param]
    weight = full[first:first + V * D].view(V, D)
    before = u.grads.clone()
    total = head(hidden, **given)
    torch.cuda.synchronize()

    def flat(name):
        x = given.get(name)
        return None if x is None else x.view(N * T, *x.shape[2:])
    kind = dict(targets=flat("targets"), index=flat("index"), teacher=flat("teacher"),
                tau=given.get("temperature", 1.0))
    ref = reference(hidden.view(N * T, D), weight, **kind, scale=float(N))
    got = dict(loss=head.loss.view(-1), lse=head.lse.view(-1), total=total,
               d_hidden=head.d_hidden.view(N * T, D))
    assert outside(got, ref) == {}
    # each rank's own part of the weight's gradient: its tokens, the total of all
    mass = float(ref["total"][0][1])
    for r in range(N):
        part = {x: y if x == "tau" or y is None else y.view(N, T, *y.shape[1:])[r]
                for x, y in kind.items()}
        one = reference(hidden[r], weight, **part, scale=N / mass, mean=False)
        mine = u.grads[r, first:first + V * D].view(V, D)
        assert outside(dict(d_weight=mine), one) == {}
    rest = torch.ones(u.grads.shape[1], dtype=torch.bool, device="cuda")
    rest[first:first + V * D] = False
    assert torch.equal(u.grads[:, rest], before[:, rest])


@pytest.mark.parametrize("k", [0, 6])
@pytest.mark.parametrize("resident", [False, True])
@pytest.mark.parametrize("lead", [(), ((24,), (16, 8))])
def test_loss_and_gradients_of_all_ranks(sch, k, resident, lead):
    model = sch.Model(units(sch, resident, lead), torch.device("cuda"))
    head = model.head(T, unit=0, param=len(lead), k=k)
    hidden, given = batch(k)
    check(sch, model, head, hidden, given, len(lead))
    # without gradients nothing but the loss changes
    kept, d = model.units[0].grads.clone(), head.d_hidden.clone()
    loss = head.loss.clone()
    head.loss.fill_(7.0)
    head(hidden, **given, grads=False)
    torch.cuda.synchronize()
    assert torch.equal(head.loss, loss) and torch.equal(head.d_hidden, d)
    assert torch.equal(model.units[0].grads, kept)


def state(model):
    return [x.clone() for u in model.units for x in (u.shards, u.master, u.m, u.v)]


@pytest.mark.parametrize("prefetch", [0, 1])
@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("max_norm", [None, 0.05])
def test_step_with_its_loss(sch, prefetch, hooked, max_norm):
    """step(loss=...) updates with the loss's gradients: two steps leave what the
    same steps leave on gradients that were put in place by hand."""
    def model():
        us, dev = units(sch), torch.device("cuda")
        return sch.PrefetchModel(us, dev, prefetch) if prefetch else sch.Model(us, dev)
    a, b = model(), model()
    hidden, given = batch()
    head, by_hand = a.head(T), b.head(T)
    seen = []
    how = dict(on_gather=lambda phase, i: seen.append((phase, i))) if hooked else {}
    for _ in range(2):
        a.step(HP, max_norm=max_norm, loss=lambda s: (seen.append("loss"),
                                                      head(hidden, **given, stream=s)), **how)
        by_hand(hidden, **given)
        torch.cuda.synchronize()
        b.step(HP, max_norm=max_norm)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert torch.equal(head.loss, by_hand.loss)
    if hooked:
        n = len(a.units)
        assert seen[:n + 2] == [("forward", i) for i in range(n)] + ["loss", ("backward", n - 1)]


def test_on_a_side_stream_first(sch):
    """The first call is on another stream than the one that the buffers were
    allocated on, whose work before them is still running."""
    model = sch.Model(units(sch), torch.device("cuda"))
    hidden, given = batch()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spin = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        spin = spin @ spin
    head = model.head(T)
    side.wait_stream(torch.cuda.current_stream())
    head(hidden, **given, stream=side)
    side.synchronize()
    first = head.loss.clone()
    other = model.head(T)
    other(hidden, **given)
    torch.cuda.synchronize()
    assert torch.equal(first, other.loss)


def test_a_captured_step_with_its_loss(sch):
    a, b = (sch.Model(units(sch), torch.device("cuda")) for _ in range(2))
    hidden, given = batch()
    ha, hb = a.head(T), b.head(T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(HP, t=1, loss=lambda s: ha(hidden, **given, stream=s))
    for _ in range(2):
        g.replay()
        b.step(HP, t=1, loss=lambda s: hb(hidden, **given, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))


def test_refusals(sch):
    model = sch.Model(units(sch), torch.device("cuda"))
    hidden, given = batch()
    head = model.head(T)
    with pytest.raises(ValueError, match="targets, or teacher"):
        head(hidden)
    with pytest.raises(ValueError, match="targets, or teacher"):
        head(hidden, **given, teacher=hidden, index=hidden)
    with pytest.raises(ValueError, match="targets: needs shape"):
        head(hidden, targets=given["targets"][:, 1:])
    with pytest.raises(ValueError, match="hidden: must be contiguous"):
        head(hidden.transpose(0, 1).contiguous().transpose(0, 1), **given)
    with pytest.raises(ValueError, match=r"not \[vocab, dim\]"):
        model.head(T, unit=1, param=4)
