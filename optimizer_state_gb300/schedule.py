"""Multi-layer ZeRO-3 step: the schedule of "The ZeRO-3 Diagram Most People
Remember Is Wrong", s.3 over a whole model.

Forward: AllGather of every unit (layer, bucket of layers or embedding) in
order.  Backward: for every unit in reverse order, AllGather again, then the
fused reduce-scatter + Adam of that unit ("ZeRO Stage 3: Parameter
Partitioning": the backward pass traverses layers in reverse).  Every gather
lands in one transient buffer sized for the largest unit (same page: the
transient buffer is bounded by the largest single layer); with prefetch
depth D there are D + 1 of them.  A resident unit (persistence threshold) is
never gathered before use: its kept copy is refreshed after its update.

The library schedules the step itself (z3_model_step); the call-by-call form
(``step(..., on_gather=hook)``) issues the same schedule from Python so that
a caller can run its own work where a unit's compute would sit.  Argument
marshalling and launch ordering only; every step runs in the CUDA library
through :mod:`optimizer_state_gb300.z3`.
"""
from __future__ import annotations

import torch

from . import inputs as I
from . import z3


class Unit:
    """Sharded state of one unit (a layer or the embedding)."""

    def __init__(self, w: I.Workload, dev, gen: torch.Generator | None, grads: bool = True,
                 hp: dict | None = None):
        self.w = w
        self.hp = hp                    # this unit's own hyperparameters (None: the step's)
        self.L = z3.Layout(w.numel, w.n_ranks)
        T = self.L.psi_padded
        self.shards = torch.empty(T, dtype=torch.bfloat16, device=dev)
        self.master = torch.empty(T, dtype=torch.float32, device=dev)
        self.m = torch.empty(T, dtype=torch.float32, device=dev)
        self.v = torch.empty(T, dtype=torch.float32, device=dev)
        self.grads = None
        # a resident unit keeps its gathered parameters for the whole run
        self.resident = torch.empty(self.L.psi, dtype=torch.bfloat16, device=dev) \
            if w.resident else None
        if gen is not None:
            full = I.draw_master(w, gen, dev).to(dev)
            self._partition(full)
            del full
            if grads:
                self.grads = I.draw_grads(w, gen, dev).to(dev)

    def _partition(self, full: torch.Tensor):
        z3.z3_partition(self.L, full, self.shards, self.master, self.m, self.v)
        if self.resident is not None:
            z3.z3_allgather(self.L, self.shards, self.resident)

    @classmethod
    def from_full(cls, w: I.Workload, dev, master_full: torch.Tensor, grads_full: torch.Tensor):
        """A unit built from given values: master_full is this unit's fp32
        parameters [Psi_u]; grads_full holds its per-rank gradients as the
        columns of a [N][>= Psi_u] tensor."""
        u = cls(w, dev, None, grads=False)
        u._partition(master_full.contiguous())
        u.grads = torch.zeros((w.n_ranks, w.grad_stride), dtype=torch.bfloat16, device=dev)
        u.grads[:, :w.psi].copy_(grads_full)
        return u

    @property
    def step_bytes(self) -> int:
        st = self.L.stats()
        # a resident unit is gathered once per step instead of twice
        return st["hbm_step_layer"] - (st["hbm_allgather"] if self.resident is not None else 0)


class Head:
    """A model's loss over the vocabulary of one of its parameters, for all of
    its logical ranks, with the gradients that a step begins from.

    A call gathers the parameter's unit (a resident one is at hand), takes the
    loss of every rank's tokens against the gathered copy in one forward pass,
    and each rank's gradients: that of the weight into the parameter's part of
    the rank's row of the unit's gradients, that of the hidden states into
    `d_hidden`.  Both are written: what else adds to the weight's gradient, such
    as a tied embedding's look-ups, is added after the call.  They are the gradients of the mean over all ranks' tokens that
    count, times the number of ranks: the step's reduction divides by it."""

    def __init__(self, model: Model, tokens: int, unit: int = 0, param: int = 0, k: int = 0):
        self.model, self.unit, self.k = model, model.units[unit], k
        u = self.unit
        shape = u.w.shapes[param]
        if len(shape) != 2:
            raise ValueError(f"parameter {param} of unit {unit} is {list(shape)}, not "
                             "[vocab, dim]")
        self.vocab, self.dim = shape
        self.tokens, self.ranks = tokens, u.w.n_ranks
        first = u.L.full_off[param]
        if first % 8 or self.dim % 8:
            what = (f"starts at element {first}" if first % 8
                    else f"has rows of {self.dim} elements")
            raise ValueError(f"parameter {param} of unit {unit} {what}: a head's weight and "
                             "its rows start on 16 bytes, a multiple of 8 elements")
        self._part = slice(first, first + self.vocab * self.dim)
        rows, dev = (self.ranks, tokens), model.dev
        self._home = torch.cuda.current_stream()   # where the buffers are allocated
        self._waited, self._seen = False, {self._home.cuda_stream}
        self.loss = torch.empty(rows, dtype=torch.float32, device=dev)
        self.lse = torch.empty(rows, dtype=torch.float32, device=dev)
        self.total = torch.empty(2, dtype=torch.float32, device=dev)
        self.d_hidden = torch.empty((*rows, self.dim), dtype=torch.bfloat16, device=dev)
        # the forward pass over all ranks, the gradients rank by rank
        need = [z3.head_workspace(n, self.dim, self.vocab, k, grads, dev)
                for n, grads in ((self.ranks * tokens, False), (tokens, True))]
        self._workspace = max(need, key=lambda x: x.numel())

    def __call__(self, hidden: torch.Tensor, targets: torch.Tensor | None = None, *,
                 teacher: torch.Tensor | None = None, index: torch.Tensor | None = None,
                 temperature: float = 1.0, weights: torch.Tensor | None = None,
                 scale: float = 1.0, grads: bool = True, stream=None) -> torch.Tensor:
        """hidden: bf16 [ranks, tokens, dim]; either targets [ranks, tokens], or
        a teacher's logits [ranks, tokens, k] with their words, index; weights:
        fp32 [ranks, tokens] or None.  Leaves loss, lse and total, and unless
        `grads` is false the gradients of scale times the mean; returns total,
        {sum of weighted losses, sum of weights} over all ranks."""
        if (targets is None) == (teacher is None) or (teacher is None) != (index is None):
            raise ValueError("give targets, or teacher and index")
        rows = (self.ranks, self.tokens)
        for x, name, tail in ((hidden, "hidden", (self.dim,)), (targets, "targets", ()),
                              (teacher, "teacher", (self.k,)), (index, "index", (self.k,)),
                              (weights, "weights", ())):
            if x is not None and tuple(x.shape) != rows + tail:
                raise ValueError(f"{name}: needs shape {list(rows + tail)}, has {list(x.shape)}")
            if x is not None and not x.is_contiguous():
                raise ValueError(f"{name}: must be contiguous")
        self._await(stream)
        u = self.unit
        full = u.resident
        if full is None:
            full = self.model.full
            z3.z3_allgather(u.L, u.shards, full, stream=stream)
        weight = full[self._part].view(self.vocab, self.dim)
        if teacher is None:
            forward, backward, heads = z3.z3_xent, z3.z3_xent_grad, (targets,)
            extra = ()
        else:
            forward, backward, heads = z3.z3_distill, z3.z3_distill_grad, (teacher, index)
            extra = (temperature,)
        forward(hidden.flatten(0, 1), weight, *[x.flatten(0, 1) for x in heads],
                *extra, self.loss.view(-1), self.lse.view(-1), self.total, self._workspace,
                weights=None if weights is None else weights.view(-1), stream=stream)
        for r in range(self.ranks if grads else 0):
            backward(hidden[r], weight, *[x[r] for x in heads], *extra, self.lse[r], self.total,
                     scale * self.ranks, self.d_hidden[r],
                     u.grads[r, self._part].view(self.vocab, self.dim), self._workspace,
                     weights=None if weights is None else weights[r], stream=stream)
        return self.total

    def _await(self, stream):
        """The first call on another stream than the one that the buffers were
        allocated on waits for that one; a captured call, which cannot wait for
        what is outside its capture, leaves it to the next.  And the allocator
        hears of each torch stream that uses them, so that a head may go while
        its calls still run.  A raw handle's stream may be gone by then: who gives
        one keeps the head until the calls have ended, as for a graph that holds
        them."""
        s = _torch_stream(stream)
        if s.cuda_stream not in self._seen and not isinstance(stream, int):
            for x in (self.loss, self.lse, self.total, self.d_hidden, self._workspace):
                x.record_stream(s)
            self._seen.add(s.cuda_stream)
        if self._waited:
            return
        if s.cuda_stream != self._home.cuda_stream:
            with torch.cuda.stream(s):
                if torch.cuda.is_current_stream_capturing():
                    return
            s.wait_stream(self._home)
        self._waited = True


class Model:
    """All units of a model plus the shared transient gathered buffer."""

    def __init__(self, units: list[Unit], dev):
        self.units = units
        self.dev = dev
        self.full = torch.empty(max([u.L.psi for u in units if u.resident is None] or [1]),
                                dtype=torch.bfloat16, device=dev)
        self.t = 0
        self.clip = None                # [norm, coef] of the last clipped step
        self._clip_args = None
        self._clip_stream = None        # where they were allocated, until a step has used them

    @property
    def psi(self) -> int:
        return sum(u.L.psi for u in self.units)

    @property
    def step_bytes(self) -> int:
        """HBM bytes of a step that is not clipped; a clipped one moves 8 more
        per padded element (the fp32 gradient, stored and read back)."""
        return sum(u.step_bytes for u in self.units)

    def head(self, tokens: int, unit: int = 0, param: int = 0, k: int = 0) -> Head:
        """The loss of `tokens` tokens of every rank over the vocabulary of one
        parameter, [vocab, dim] (an embedding's where the head is tied to it),
        whose dim and place in its unit are multiples of 8 elements; k: the
        length of a teacher's lists, where there is one."""
        return Head(self, tokens, unit, param, k)

    def launches_per_step(self) -> int:
        """Kernel launches of a step that is not clipped."""
        n = 0
        for u in self.units:
            tabs = -(-sum(1 for x in u.L.numel if x > 0) // 40)
            n += (2 if u.resident is not None else 3) * tabs
        return n

    def unit_args(self):
        return [(u.L, u.shards, u.master, u.m, u.v, u.grads, u.w.grad_stride,
                 1.0 / u.w.n_ranks, u.resident, u.hp) for u in self.units]

    def clip_args(self, stream=None):
        """What a clipped step keeps beside the units' state: for each unit its
        reduced fp32 gradient and its sums of squares, and for all of them
        the norm's list and workspace and [norm, coef].  Allocated and zeroed
        by the first call, in the order of `stream` (None: the current one):
        by the first clipped step on its own stream, or by a call before it.
        A step that is to be captured wants that call first, or its graph
        holds the zeroing too."""
        if self._clip_args is None:
            self._clip_stream = _torch_stream(stream)
            with torch.cuda.stream(self._clip_stream):
                self._clip_args = [
                    (torch.zeros(u.L.psi_padded, dtype=torch.float32, device=self.dev),
                     torch.zeros(u.L.sumsq_len, dtype=torch.float64, device=self.dev))
                    for u in self.units]
                self._sums = z3.TensorList([], sumsq=[sq for _, sq in self._clip_args])
                self._workspace = z3.grad_norm_workspace(self.dev)
                self.clip = torch.zeros(2, dtype=torch.float32, device=self.dev)
        return self._clip_args

    def _step_clip_args(self, stream):
        """clip_args() for a step on `stream`.  The first step waits there for
        the stream that they were allocated on, where that is another: the
        zeroing, and whatever used that memory before, come first.  A capture
        cannot wait for what is outside it (its graph runs after what its
        capture came after), so the wait is left to the next step."""
        clips = self.clip_args(stream)
        if self._clip_stream is not None:
            s = _torch_stream(stream)
            if s.cuda_stream != self._clip_stream.cuda_stream:
                with torch.cuda.stream(s):
                    if torch.cuda.is_current_stream_capturing():
                        return clips
                s.wait_stream(self._clip_stream)
            self._clip_stream = None
        return clips

    def _library_step(self, full, hp: dict, t: int, max_norm, stream, gather_stream=None):
        if max_norm is None:
            z3.z3_model_step(self.unit_args(), full, hp, t, stream=stream,
                             gather_stream=gather_stream)
        else:
            clips = self._step_clip_args(stream)
            z3.z3_model_step_clipped(self.unit_args(), clips, full, hp, t, max_norm, self.clip,
                                     self._workspace, stream=stream, gather_stream=gather_stream)

    def _take_loss(self, loss, stream, counted: bool):
        if loss is None:
            return
        try:
            loss(stream)
        except Exception:
            self.t -= counted
            raise

    def _backward(self, i: int, hp: dict, t: int, max_norm, stream):
        """What follows the backward compute of unit i: its update, or in a
        clipped step its reduced gradient and sums of squares."""
        u = self.units[i]
        if max_norm is None:
            self._update(u, hp, t, stream)
        else:
            gs, sq = self._step_clip_args(stream)[i]
            z3.z3_reduce_scatter_norm(u.L, u.grads, u.w.grad_stride, gs, 1.0 / u.w.n_ranks, sq,
                                      stream=stream)

    def _finish(self, hp: dict, t: int, max_norm, stream):
        """The rest of a clipped step, once every unit is reduced: the calls of
        z3_model_step_clipped, but for its one launch of all updates (24
        layers and an embedding: 3.90 ms issued from here, 3.73 there)."""
        if max_norm is None:
            return
        z3.z3_grad_norm(self._sums, max_norm, self.clip, self._workspace, stream=stream)
        for u, (gs, _) in zip(self.units, self.clip_args()):
            z3.z3_adam_shard_step_clipped(u.L, u.master, u.m, u.v, gs, u.shards, u.hp or hp, t,
                                          self.clip, stream=stream)
            if u.resident is not None:
                z3.z3_allgather(u.L, u.shards, u.resident, stream=stream)

    @staticmethod
    def _update(u: Unit, hp: dict, t: int, stream):
        z3.z3_reduce_scatter_adam(u.L, u.grads, u.w.grad_stride, 1.0 / u.w.n_ranks, None,
                                  u.master, u.m, u.v, u.shards, u.hp or hp, t, stream=stream)
        if u.resident is not None:
            z3.z3_allgather(u.L, u.shards, u.resident, stream=stream)

    def step(self, hp: dict, stream=None, t: int | None = None, on_gather=None,
             max_norm: float | None = None, loss=None):
        """One training step, scheduled by the library (z3_model_step).
        `loss(stream)` is called where the backward pass begins, such as for a
        Head's call: after the forward gathers of a step with hooks, and before
        a step that the library schedules as a whole.  Where it raises, no state
        has been touched and the step keeps no number.
        With `max_norm` the gradients of all units are clipped to that global
        norm first (z3_model_step_clipped); `clip` then holds [norm, coef] on
        the device, coef NaN where the norm was not finite and the step was
        left out (it keeps its number: the host does not know of it; a caller
        that reads `clip` may pass the same `t` again).  That takes 4 more
        bytes per element (the fp32 gradients).
        With `on_gather(phase, index)` the same schedule is issued call by
        call from here instead, and the hook is called after each gather is
        enqueued, with the transient buffer holding that unit's parameters
        once the stream reaches it -- the point where the forward or backward
        compute of the unit would run."""
        counted = t is None
        if counted:
            self.t += 1
            t = self.t
        if on_gather is None:
            self._take_loss(loss, stream, counted)
            self._library_step([self.full], hp, t, max_norm, stream)
            return
        for i, u in enumerate(self.units):            # forward
            if u.resident is None:
                z3.z3_allgather(u.L, u.shards, self.full, stream=stream)
            on_gather("forward", i)
        self._take_loss(loss, stream, counted)
        for i in range(len(self.units) - 1, -1, -1):    # backward, reverse order
            u = self.units[i]
            if u.resident is None:
                z3.z3_allgather(u.L, u.shards, self.full, stream=stream)
            on_gather("backward", i)
            self._backward(i, hp, t, max_norm, stream)
        self._finish(hp, t, max_norm, stream)


def _torch_stream(stream):
    """A torch stream object for a stream argument (None: the current stream;
    an int: a raw cudaStream_t handle).  Handle 0 is the legacy default
    stream; torch's stream wrapper treats a zero pointer as "none given" and
    hands out a fresh pool stream instead, which would leave the work
    unordered with everything else on the default stream, so 0 maps to
    torch's default stream explicitly."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, int):
        return torch.cuda.default_stream() if stream == 0 else torch.cuda.ExternalStream(stream)
    return stream


class PrefetchModel(Model):
    """The same step with the gather of the next unit prefetched one unit
    ahead on a second stream ("ZeRO Stage 3: Parameter Partitioning": the
    All-Gather for layer l+1 proceeds while layer l computes; "ZeRO Stages:
    ...": prefetched layers occupy memory, so two transient buffers).

    Backward: the gather of unit i-1 runs on the gather stream while unit i's
    fused reduce-scatter + Adam runs on the main stream.  Ordering is by
    events: a unit's update waits for its gather; a gather into a buffer waits
    until the update of the unit that last used that buffer is enqueued after
    it (the point where that unit's backward compute would have finished)."""

    def __init__(self, units: list[Unit], dev, depth: int = 1):
        super().__init__(units, dev)
        self.depth = depth
        self.bufs = [self.full] + [torch.empty_like(self.full) for _ in range(depth)]
        self.gstream = torch.cuda.Stream(device=dev)

    def step(self, hp: dict, stream=None, t: int | None = None, on_gather=None,
             max_norm: float | None = None, loss=None):
        counted = t is None
        if counted:
            self.t += 1
            t = self.t
        if on_gather is None:
            self._take_loss(loss, stream, counted)
            self._library_step(self.bufs, hp, t, max_norm, stream, self.gstream)
            return
        if self.depth != 1:
            raise NotImplementedError("the call-by-call schedule prefetches one unit ahead")
        main = _torch_stream(stream)
        g = self.gstream
        n = len(self.units)
        freed = [torch.cuda.Event(), torch.cuda.Event()]
        g.wait_stream(main)                            # shards updated by the last step
        for i, u in enumerate(self.units):            # forward, back to back on g
            if u.resident is None:
                z3.z3_allgather(u.L, u.shards, self.bufs[i % 2], stream=g.cuda_stream)
            with torch.cuda.stream(g):
                on_gather("forward", i)
        with torch.cuda.stream(g):
            self._take_loss(loss, g, counted)
        order = list(range(n - 1, -1, -1))
        gathered = {}

        def gather(i):
            u = self.units[i]
            if u.resident is None:
                z3.z3_allgather(u.L, u.shards, self.bufs[i % 2], stream=g.cuda_stream)
            with torch.cuda.stream(g):
                on_gather("backward", i)
            ev = torch.cuda.Event()
            ev.record(g)
            gathered[i] = ev
        gather(order[0])
        for k, i in enumerate(order):
            u = self.units[i]
            if k + 1 < n:
                nxt = order[k + 1]
                if k >= 1:
                    g.wait_event(freed[nxt % 2])       # buffer of unit i+1 is free again
                gather(nxt)                            # prefetch one unit ahead
            main.wait_event(gathered[i])
            self._backward(i, hp, t, max_norm, main.cuda_stream)
            freed[i % 2].record(main)
        main.wait_stream(g)
        self._finish(hp, t, max_norm, main.cuda_stream)


def full_step_model(dev, seed: int = 0, prefetch: int = 0, bucket_layers: int = 1,
                    persistence_threshold: int = 0) -> Model:
    """The 24-layer d=1024 model with its [50257, 1024] embedding, N_d = 16.

    bucket_layers: the parameter-bucket knob of "The ZeRO-3 Diagram Most
    People Remember Is Wrong", s.8 -- that many consecutive layers form one
    unit (one gather and one fused reduce-scatter + Adam launch each; the
    transient buffer grows to the largest unit).  Every parameter is still
    partitioned on its own, and the update is elementwise, so the result of
    a step does not depend on the bucket size.

    prefetch: how many units ahead the backward gathers run on a second stream
    (0: none; each unit of depth costs one more transient buffer).

    persistence_threshold: the persistence-threshold knob of the same section
    -- parameters of fewer elements are not released after use: they form
    one resident unit whose gathered copy is kept and refreshed once per step
    after its update, instead of being gathered before every use.
    """
    gen = I.make_generator(seed, dev)
    units = [Unit(w, dev, gen) for w in I.full_step_units(bucket_layers, persistence_threshold)]
    return PrefetchModel(units, dev, int(prefetch)) if prefetch else Model(units, dev)



# ---------------------------------------------------------------------------
# The other ZeRO stages and plain data parallelism on the same kernels
# ("ZeRO Stages: Sharding Optimizer State, Gradients, and Parameters";
# "ZeRO Stage 3: Parameter Partitioning", communication list).  Each returns
# the HBM bytes per unpadded element its launches move.
# ---------------------------------------------------------------------------

def stage2_step(u: Unit, full: torch.Tensor, hp: dict, t: int, stream=None) -> int:
    """Stage 2: reduce-scatter the gradients (fused with the shard Adam), then
    one all-gather of the updated parameters into the replica."""
    N = u.w.n_ranks
    z3.z3_reduce_scatter_adam(u.L, u.grads, u.w.grad_stride, 1.0 / N, None, u.master, u.m, u.v,
                              u.shards, hp, t, stream=stream)
    z3.z3_allgather(u.L, u.shards, full, stream=stream)
    return (2 * N + 26) + 4


def stage1_step(u: Unit, grad_full: torch.Tensor, grad_shards: torch.Tensor,
                full: torch.Tensor, hp: dict, t: int, stream=None) -> int:
    """Stage 1: all-reduce the gradients (every rank receives the full sum),
    each rank updates its slice of the optimizer state from its slice of the
    reduced gradient, then an all-gather of the updated parameters."""
    N = u.w.n_ranks
    z3.z3_allreduce(u.L, u.grads, u.w.grad_stride, grad_full, 1.0 / N, stream=stream)
    z3.z3_scatter(u.L, grad_full, grad_shards, stream=stream)
    z3.z3_adam_shard_step(u.L, u.master, u.m, u.v, grad_shards, u.shards, hp, t, stream=stream)
    z3.z3_allgather(u.L, u.shards, full, stream=stream)
    return (2 * N + 4) + 8 + 30 + 4


class DPReplica:
    """Plain data parallelism: every rank holds the whole fp32 master, m, v and
    bf16 parameters; the state is laid out as one rank (N = 1)."""

    def __init__(self, w: I.Workload, dev, gen: torch.Generator):
        self.w = w
        self.L = z3.Layout(w.numel, w.n_ranks)         # the gradient fold over N ranks
        self.L1 = z3.Layout(w.numel, 1)                # unsharded state
        n = self.L1.psi
        self.params = torch.empty(n, dtype=torch.bfloat16, device=dev)
        self.master = torch.empty(n, dtype=torch.float32, device=dev)
        self.m = torch.empty(n, dtype=torch.float32, device=dev)
        self.v = torch.empty(n, dtype=torch.float32, device=dev)
        full = I.draw_master(w, gen, dev).to(dev)
        z3.z3_partition(self.L1, full, self.params, self.master, self.m, self.v)
        self.grads = I.draw_grads(w, gen, dev).to(dev)
        self.grad_full = torch.empty(n, dtype=torch.float32, device=dev)

    def step(self, hp: dict, t: int, stream=None) -> int:
        N = self.w.n_ranks
        z3.z3_allreduce(self.L, self.grads, self.w.grad_stride, self.grad_full, 1.0 / N,
                        stream=stream)
        z3.z3_adam_shard_step(self.L1, self.master, self.m, self.v, self.grad_full, self.params,
                              hp, t, stream=stream)
        return (2 * N + 4) + 30
