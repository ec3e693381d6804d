"""The losses over a vocabulary on the CPU: what their entry points refuse, with
the status and the words of each refusal, the workspace's size, the structures'
layout, and what the binding refuses.  Made-up device addresses are only used in
a child process that sees no device."""
import ctypes
import math
import subprocess

import pytest
import torch

from optimizer_state_gb300 import build as z3build
from optimizer_state_gb300 import z3

A = 1 << 32                       # an aligned made-up address
INV, ALI, OVF = z3.Z3_ERR_INVALID_ARG, z3.Z3_ERR_ALIGNMENT, z3.Z3_ERR_OVERFLOW


@pytest.fixture(scope="module")
def lib():
    z3build.build()
    return z3.load()


def test_structs_are_laid_out_as_in_the_header(tmp_path):
    fields = {"z3_head": z3.Head, "z3_teacher": z3.Teacher}
    lines = [f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {f}));'
             for n, c in fields.items() for f, _ in c._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "z3.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{z3build.INCLUDE}", str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    want = [x for c in fields.values() for f, _ in c._fields_
            for x in (ctypes.sizeof(c), getattr(c, f).offset)]
    assert list(map(int, got)) == want


def size(lib, tokens, dim, vocab, k=0, grads=1):
    n = ctypes.c_int64(-1)
    st = lib.z3_head_workspace_bytes(tokens, dim, vocab, k, grads, ctypes.byref(n))
    return st, n.value


def test_workspace(lib):
    assert lib.z3_head_workspace_bytes(1, 8, 1, 0, 1, None) == INV
    for args, status in (((-1, 8, 1), INV), ((1, 0, 1), INV), ((1, 12, 1), INV), ((1, 8, 0), INV),
                         ((1, 8, 1, -1), INV), ((1, 8, 1, 1025), INV),
                         ((2 ** 31, 8, 1), OVF), ((1, 8, 2 ** 31), OVF), ((1, 2 ** 31, 1), OVF),
                         ((2 ** 31 - 1024, 8, 2 ** 31 - 1024), OVF)):
        st, n = size(lib, *args)
        assert (st, n) == (status, -1), args
    # the forward pass alone takes less; dz takes a piece of the vocabulary at a time
    forward, both = (size(lib, 8192, 1024, 50257, 0, g)[1] for g in (0, 1))
    assert forward < both < 600 << 20
    assert size(lib, 8192, 1024, 50257, 64)[1] > both
    # never as much as the logits of a large vocabulary
    assert size(lib, 65536, 1024, 131072)[1] < 65536 * 131072 * 2 // 8
    assert size(lib, 0, 8, 1)[0] == z3.Z3_OK


class Call:
    """A call with valid made-up arguments, some of them replaced."""

    def __init__(self, lib, name, **kw):
        self.tokens, self.vocab, self.dim, self.k = 100, 300, 64, 5
        a = dict(hidden=A, hidden_stride=64, weight=A + (1 << 20), weight_stride=72, tokens=100,
                 vocab=300, dim=64, weights=A + (2 << 20), index=A + (3 << 20), index_bytes=8,
                 logits=A + (4 << 20), dtype=z3.Z3_F32, k=5, temperature=2.0,
                 loss=A + (5 << 20), lse=A + (6 << 20), total=A + (7 << 20), scale=1.0,
                 d_hidden=A + (8 << 20), d_hidden_stride=64, d_weight=A + (9 << 20),
                 d_weight_stride=64, workspace=A + (1 << 30), workspace_bytes=1 << 40, head=True,
                 teacher=True)
        assert set(kw) <= set(a)
        a |= kw
        head = z3.Head(a["hidden"], a["hidden_stride"], a["weight"], a["weight_stride"],
                       a["tokens"], a["vocab"], a["dim"], a["weights"])
        teacher = z3.Teacher(a["logits"], a["index"], a["dtype"], a["index_bytes"], a["k"],
                             a["temperature"])
        h = ctypes.byref(head) if a["head"] else None
        t = ctypes.byref(teacher) if a["teacher"] else None
        end = (a["workspace"], a["workspace_bytes"], None)
        out = (a["loss"], a["lse"], a["total"])
        grads = (a["lse"], a["total"], a["scale"], a["d_hidden"], a["d_hidden_stride"],
                 a["d_weight"], a["d_weight_stride"])
        what = (t,) if "distill" in name else (a["index"], a["index_bytes"])
        self.status = getattr(lib, name)(h, *what, *(grads if "grad" in name else out), *end)
        self.message = z3.last_error()


CALLS = ("z3_xent", "z3_xent_grad", "z3_distill", "z3_distill_grad")


@pytest.mark.no_device
@pytest.mark.parametrize("name", CALLS)
def test_refusals(lib, name):
    grad, distill = "grad" in name, "distill" in name
    index = "index" if distill else "targets"
    bad = [(dict(head=False), INV, "head is NULL"),
           (dict(hidden=None), INV, "hidden is NULL"), (dict(weight=None), INV, "weight is NULL"),
           (dict(index=None), INV, f"{index} is NULL"), (dict(lse=None), INV, "lse is NULL"),
           (dict(workspace=None), INV, "workspace is NULL"),
           (dict(hidden=A + 8), ALI, "hidden is not 16-byte"),
           (dict(weight=A + 8), ALI, "weight is not 16-byte"),
           (dict(workspace=A + (1 << 30) + 8), ALI, "workspace is not 16-byte"),
           (dict(index=A + (3 << 20) + 4), ALI, f"{index} is not 8-byte"),
           (dict(index_bytes=4, index=A + (3 << 20) + 2), ALI, f"{index} is not 4-byte"),
           (dict(weights=A + (2 << 20) + 2), ALI, "weights is not 4-byte"),
           (dict(lse=A + (6 << 20) + 2), ALI, "lse is not 4-byte"),
           (dict(index_bytes=2), INV, "index_bytes"), (dict(index_bytes=0), INV, "index_bytes"),
           (dict(tokens=-1), INV, "tokens < 0"), (dict(vocab=0), INV, "vocab < 1"),
           (dict(dim=0), INV, "dim < 1"), (dict(dim=60), INV, "multiple of 8"),
           (dict(tokens=2 ** 31), OVF, "do not fit"), (dict(vocab=2 ** 31), OVF, "do not fit"),
           (dict(hidden_stride=56), INV, "hidden_stride < dim"),
           (dict(weight_stride=66), ALI, "weight_stride is not"),
           (dict(hidden_stride=2 ** 40), OVF, "hidden does not fit"),
           (dict(workspace_bytes=4096), INV, "the workspace has 4096 bytes, needs"),
           (dict(workspace=A), INV, "workspace overlaps hidden"),
           (dict(workspace=A + (3 << 20)), INV, f"workspace overlaps {index}")]
    if grad:
        bad += [(dict(scale=math.nan), INV, "scale"), (dict(scale=math.inf), INV, "scale"),
                (dict(d_hidden=A + (8 << 20) + 2), ALI, "d_hidden is not 16-byte"),
                (dict(d_weight=A + (9 << 20) + 8), ALI, "d_weight is not 16-byte"),
                (dict(d_hidden_stride=56), INV, "d_hidden_stride < dim"),
                (dict(d_weight_stride=68), ALI, "d_weight_stride"),
                (dict(d_hidden=A), INV, "d_hidden overlaps hidden"),
                (dict(d_weight=A + (1 << 20) + 128), INV, "d_weight overlaps weight"),
                (dict(d_weight=A + (8 << 20) + 99 * 128), INV, "d_weight overlaps d_hidden"),
                (dict(d_hidden=A + (1 << 30)), INV, "d_hidden overlaps workspace"),
                (dict(total=A + (7 << 20) + 2), ALI, "total is not 4-byte")]
    else:
        bad += [(dict(loss=None), INV, "loss is NULL"), (dict(total=None), INV, "total is NULL"),
                (dict(loss=A + (6 << 20) + 396), INV, "lse overlaps loss"),
                (dict(total=A + (2 << 20)), INV, "total overlaps weights"),
                (dict(lse=A + 64), INV, "lse overlaps hidden")]
    if distill:
        bad += [(dict(teacher=False), INV, "teacher is NULL"), (dict(k=0), INV, "1..1024"),
                (dict(k=1025), INV, "1..1024"), (dict(dtype=z3.Z3_SUMSQ), INV, "logits are"),
                (dict(logits=None), INV, "logits is NULL"),
                (dict(logits=A + (4 << 20) + 2), ALI, "logits is not 4-byte"),
                (dict(dtype=z3.Z3_BF16, logits=A + (4 << 20) + 1), ALI, "logits is not 2-byte"),
                *[(dict(temperature=x), INV, "temperature")
                  for x in (0.0, -1.0, math.nan, math.inf, 1e20, 1e-39)]]
    for kw, status, words in bad:
        c = Call(lib, name, **kw)
        assert (c.status, words in c.message and c.message.startswith(name)) == (status, True), \
            (kw, c.status, c.message)
    # all in order: only the launch can fail, in a process without a device
    for kw in ({}, dict(weights=None), dict(index_bytes=4), dict(hidden_stride=128)):
        assert Call(lib, name, **kw).status == z3.Z3_ERR_CUDA
    if grad:
        assert Call(lib, name, d_hidden=None, d_weight=None).status == z3.Z3_OK   # nothing to do
        for kw in (dict(d_hidden=None), dict(d_weight=None), dict(total=None)):
            assert Call(lib, name, **kw).status == z3.Z3_ERR_CUDA


def test_the_binding_refuses_tensors_of_the_wrong_kind(lib):
    """Before it asks for their addresses: no device is needed."""
    h, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    y, f, ws = torch.zeros(4, dtype=torch.long), torch.zeros(4), torch.zeros(9, dtype=torch.uint8)
    with pytest.raises(ValueError, match="hidden: must be a CUDA tensor"):
        z3.z3_xent(h, w, y, f, f, f[:2], ws)
    with pytest.raises(ValueError, match="hidden: needs two dimensions"):
        z3.z3_xent(h[0], w, y, f, f, f[:2], ws)
    with pytest.raises(ValueError, match="weight: needs two dimensions"):
        z3.z3_distill(h, w[0], f, y, 1.0, f, f, f[:2], ws)
    for args in ((-1, 8, 1), (1, 9, 1), (1, 8, 1, 2000)):
        with pytest.raises(z3.Z3Error):
            z3.head_workspace(*args, device="cpu")
    assert z3.head_workspace(10, 8, 20, device="cpu").dtype == torch.uint8
