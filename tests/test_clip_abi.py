"""Gradient clipping on the CPU: what the entry points refuse, with the status
and the words of each refusal, and the lengths that they tell.  Made-up device
addresses are only used in a child process that sees no device."""
import ctypes
import math
import subprocess

import pytest

from optimizer_state_gb300 import build as z3build
from optimizer_state_gb300 import z3

A = 1 << 32                       # an aligned made-up address


@pytest.fixture(scope="module")
def lib():
    z3build.build()
    return z3.load()


def test_structs_are_laid_out_as_in_the_header(tmp_path):
    """The binding's structures against a C compiler's."""
    fields = {"z3_tensor": (z3.Tensor, ["data", "numel", "dtype", "reserved"]),
              "z3_clip_unit": (z3.ClipUnit, ["grad_shards", "sumsq", "accumulate", "reserved"])}
    lines = [f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {f}));'
             for n, (_, fs) in fields.items() for f in fs]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "z3.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{z3build.INCLUDE}", str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    want = [x for c, fs in fields.values() for f in fs
            for x in (ctypes.sizeof(c), getattr(c, f).offset)]
    assert list(map(int, got)) == want
    assert (z3.Z3_BF16, z3.Z3_F32, z3.Z3_SUMSQ) == (0, 1, 2)


def test_sumsq_len_counts_the_reduce_tiles(lib):
    # one sum per CTA: 128 vectors of 8 elements of one (parameter, rank) slice
    assert z3.Layout([1024 * 8], 8).sumsq_len == 8
    assert z3.Layout([1024 * 8 * 2, 64], 8).sumsq_len == 8 * 2 + 8
    # S = 2049: a slice that starts inside a vector touches 257 of them
    assert z3.Layout([1024 * 8 * 2, 8], 8).sumsq_len == 8 * 3 + 8
    assert z3.Layout([0, 0], 4).sumsq_len == 0
    assert z3.Layout([64] * 41, 8).sumsq_len == 41 * 8      # two launch tables
    n = ctypes.c_int64()
    assert lib.z3_sumsq_len(None, ctypes.byref(n)) == z3.Z3_ERR_INVALID_ARG
    assert lib.z3_sumsq_len(z3.Layout([5], 1).handle, None) == z3.Z3_ERR_INVALID_ARG
    assert lib.z3_grad_norm_workspace_bytes(None) == z3.Z3_ERR_INVALID_ARG


class List:
    """A z3_tensor_list of (address, numel, dtype) triples, and its status."""

    def __init__(self, lib, *ts, n=None):
        self.lib = lib
        arr = (z3.Tensor * len(ts))(*[z3.Tensor(*t, 0) for t in ts])
        self.h = ctypes.c_void_p(7)
        self.status = lib.z3_tensor_list_create(arr, len(ts) if n is None else n,
                                                ctypes.byref(self.h))
        self.message = z3.last_error()

    def __del__(self):
        self.lib.z3_tensor_list_destroy(self.h)


@pytest.mark.no_device
def test_tensor_list_refusals(lib):
    d = A + (1 << 30)
    ok = (d, 100, z3.Z3_F32)
    inv, ali, ovf = z3.Z3_ERR_INVALID_ARG, z3.Z3_ERR_ALIGNMENT, z3.Z3_ERR_OVERFLOW
    for ts, n, status, words in (
            ([ok], -1, inv, "n < 0"),
            ([(d, 100, 3)], None, inv, "tensors[0]: unknown dtype"),
            ([(d, 100, -1)], None, inv, "unknown dtype"),
            ([ok, (d, -1, z3.Z3_F32)], None, inv, "tensors[1]: numel"),
            ([(None, 1, z3.Z3_F32)], None, inv, "NULL"),
            ([(d + 2, 1, z3.Z3_F32)], None, ali, "tensors[0]"),
            ([ok, (d + 1, 1, z3.Z3_BF16)], None, ali, "tensors[1]"),
            ([(d + 4, 1, z3.Z3_SUMSQ)], None, ali, "tensors[0]"),
            ([(d, 1 << 62, z3.Z3_F32)], None, ovf, "tensors[0]"),
            ([(d, 1 << 60, z3.Z3_F32)], None, ovf, "tensors[0]"),   # past any address
            ([((1 << 64) - 64, 32, z3.Z3_F32)], None, ovf, "tensors[0]")):
        x = List(lib, *ts, n=n)
        assert (x.status, x.h.value) == (status, None) and words in x.message, (ts, x.message)
    h = ctypes.c_void_p()
    assert lib.z3_tensor_list_create(None, 1, ctypes.byref(h)) == inv
    assert lib.z3_tensor_list_create(None, 0, None) == inv
    assert lib.z3_tensor_list_create(None, 0, ctypes.byref(h)) == z3.Z3_OK
    lib.z3_tensor_list_destroy(h)
    lib.z3_tensor_list_destroy(None)  # no-op


@pytest.mark.no_device
def test_grad_norm_and_clip_refusals(lib):
    clip, ws = A, A + (1 << 20)
    d = A + (1 << 30)
    ok = (d, 100, z3.Z3_F32)
    inv, ali = z3.Z3_ERR_INVALID_ARG, z3.Z3_ERR_ALIGNMENT

    def norm(*ts, max_norm=1.0, clip=clip, ws=ws):
        x = List(lib, *ts)
        assert x.status == z3.Z3_OK
        return lib.z3_grad_norm(x.h, max_norm, clip, ws, None), z3.last_error()

    def scale(*ts, clip=clip):
        x = List(lib, *ts)
        assert x.status == z3.Z3_OK
        return lib.z3_clip(x.h, clip, None), z3.last_error()

    for bad in (0.0, -1.0, math.nan, -math.inf):
        s, msg = norm(ok, max_norm=bad)
        assert s == inv and "max_norm" in msg, bad
    for call in (norm, scale):
        s, msg = call(ok, clip=None)
        assert s == inv and "clip" in msg
        s, msg = call(ok, clip=clip + 4)
        assert s == ali and "clip" in msg
        s, msg = call((d, 1, z3.Z3_F32), (d + 16, 0, z3.Z3_F32), (clip + 4, 1, z3.Z3_F32))
        assert s == inv and "tensors[2] overlaps clip" in msg
    s, msg = norm(ok, ws=None)
    assert s == inv and "workspace" in msg
    s, msg = norm(ok, ws=ws + 8)
    assert s == ali and "workspace" in msg
    s, msg = norm(ok, ws=clip)
    assert s == inv and "overlaps" in msg
    s, msg = norm((ws + 16, 1, z3.Z3_BF16))
    assert s == inv and "overlaps workspace" in msg
    assert lib.z3_grad_norm(None, 1.0, clip, ws, None) == inv
    assert lib.z3_clip(None, clip, None) == inv
    s, msg = scale(ok, (d + 4096, 8, z3.Z3_SUMSQ))
    assert s == inv and "tensors[1] holds sums of squares" in msg
    # overlapping tensors, in ascending and in other orders
    s, msg = scale(ok, (d + 396, 4, z3.Z3_F32))
    assert s == inv and "tensors[1] overlaps tensors[0]" in msg
    s, msg = scale((d + 396, 4, z3.Z3_F32), ok)
    assert s == inv and "overlaps" in msg
    s, msg = scale((None, 0, z3.Z3_F32), (d + 4096, 4, z3.Z3_F32), ok, (d + 398, 1, z3.Z3_BF16))
    assert s == inv and "tensors[3] overlaps tensors[2]" in msg
    # what is right gets as far as the launch, which finds no device
    assert norm(ok, ok, (None, 0, z3.Z3_F32), (d + 2, 1, z3.Z3_BF16))[0] == z3.Z3_ERR_CUDA
    assert scale((d + 400, 4, z3.Z3_F32), ok)[0] == z3.Z3_ERR_CUDA


@pytest.mark.no_device
def test_reduce_scatter_norm_and_clipped_adam_refusals(lib):
    L = z3.Layout([35, 13, 12], 4)
    far = A + (1 << 28)
    inv, ali = z3.Z3_ERR_INVALID_ARG, z3.Z3_ERR_ALIGNMENT

    def st(s):
        return s, z3.last_error()

    sq = far + (1 << 20)
    assert lib.z3_reduce_scatter_norm(None, A, 64, far, 0.25, 0, sq, None) == inv
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 61, far, 0.25, 0, sq, None))
    assert s == ali
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 56, far, 0.25, 0, sq, None))
    assert s == inv and "grad_stride" in msg
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 64, far, math.inf, 0, sq, None))
    assert s == inv and "scale" in msg
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 64, far, 0.25, 0, None, None))
    assert s == inv and "sumsq" in msg
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 64, far, 0.25, 0, sq + 8, None))
    assert s == ali and "sumsq" in msg
    s, msg = st(lib.z3_reduce_scatter_norm(L.handle, A, 64, far, 0.25, 0, far + 16, None))
    assert s == inv and "overlaps" in msg

    hp = z3.AdamHP(1e-3, 0.9, 0.999, 1e-8, 0.0)
    bufs = [A + i * (1 << 24) for i in range(6)]

    def adam(b=bufs[:5], hp=hp, step=1, clip=bufs[5]):
        return st(lib.z3_adam_shard_step_clipped(L.handle, *b, ctypes.byref(hp), step, clip, None))

    assert adam(step=0)[0] == inv
    assert adam(hp=z3.AdamHP(math.nan, 0.9, 0.999, 1e-8, 0.0))[0] == inv
    s, msg = adam(clip=None)
    assert s == inv and "clip" in msg
    s, msg = adam(clip=bufs[5] + 4)
    assert s == ali and "clip" in msg
    s, msg = adam(clip=bufs[2])
    assert s == inv and "overlaps" in msg
    assert lib.z3_adam_shard_step_clipped(None, *bufs[:5], ctypes.byref(hp), 1, bufs[5],
                                          None) == inv
    # an empty layer is a no-op
    E = z3.Layout([0], 4)
    assert lib.z3_reduce_scatter_norm(E.handle, None, 0, None, 1.0, 0, None, None) == z3.Z3_OK
    assert lib.z3_adam_shard_step_clipped(E.handle, *[None] * 5, ctypes.byref(hp), 1, bufs[5],
                                          None) == z3.Z3_OK


@pytest.mark.no_device
def test_clipped_model_step_refusals(lib):
    L = z3.Layout([1000], 4)
    inv, ali = z3.Z3_ERR_INVALID_ARG, z3.Z3_ERR_ALIGNMENT
    hp = z3.AdamHP(1e-3, 0.9, 0.999, 1e-8, 0.0)
    at = iter(range(A, 1 << 40, 1 << 20))
    units = (z3.Unit * 2)(*[z3.Unit(L.handle.value, next(at), next(at), next(at), next(at),
                                    next(at), 1000, 0.25, None, None) for _ in range(2)])
    good = [[next(at), next(at)] for _ in range(2)]
    full, clip, ws = next(at), next(at), next(at)

    def step(units=units, clips=good, full=full, clip=clip, ws=ws, max_norm=1.0, n=2,
             null_clips=False):
        carr = None if null_clips else (z3.ClipUnit * 2)(*[z3.ClipUnit(*c, 0, 0) for c in clips])
        fulls = (ctypes.c_void_p * 1)(full)
        return lib.z3_model_step_clipped(units, carr, n, fulls, 1, ctypes.byref(hp), 1, max_norm,
                                         clip, ws, None, None), z3.last_error()

    s, msg = step(null_clips=True)
    assert s == inv and "clips" in msg
    s, msg = step(n=0)
    assert s == inv and "z3_model_step_clipped" in msg
    s, msg = step(max_norm=0.0)
    assert s == inv and "max_norm" in msg
    for name in ("clip", "ws"):
        s, msg = step(**{name: None})
        assert s == inv
        s, msg = step(**{name: good[0][0] + 4})
        assert s == ali
    for i in (0, 1):
        s, msg = step(clips=[[None, c[1]] if k == i else c for k, c in enumerate(good)])
        assert s == inv and "grad_shards" in msg
        s, msg = step(clips=[[c[0], None] if k == i else c for k, c in enumerate(good)])
        assert s == inv and "sumsq" in msg
    # every pair of buffers that must be apart
    for what, kw in (("sumsq", dict(clips=[[good[0][0], good[0][0]], good[1]])),
                     ("sumsq", dict(clips=[good[0], [good[1][0], good[0][1]]])),
                     ("grad_shards", dict(clips=[good[0], [good[0][0] + 16, good[1][1]]])),
                     ("grad_shards", dict(clips=[[units[1].grads, good[0][1]], good[1]])),
                     ("grad_shards", dict(clips=[[units[0].m, good[0][1]], good[1]])),
                     ("sumsq", dict(clips=[[good[0][0], units[0].shards], good[1]])),
                     ("sumsq", dict(clips=[[good[0][0], full], good[1]])),
                     ("clip", dict(clip=units[1].master)), ("clip", dict(clip=full)),
                     ("clip", dict(clip=ws)), ("workspace", dict(ws=good[1][1])),
                     ("workspace", dict(ws=full))):
        s, msg = step(**kw)
        assert s == inv and "overlaps" in msg and what in msg, (kw, msg)
    assert step()[0] == z3.Z3_ERR_CUDA          # all right: no device to launch on


def test_bindings_refuse_host_tensors():
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        z3.TensorList([torch.zeros(3)])
    with pytest.raises(ValueError, match="clips"):
        z3.z3_model_step_clipped([1, 2], [1], [], {}, 1, 1.0, None, None)
