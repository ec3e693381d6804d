"""Thin ctypes binding of the C ABI in ``include/z3.h``.

Argument marshalling only: every step of the path runs in the CUDA library
``_build/libz3.so``.  Functions keep the C names; device buffers may be
passed as CUDA tensors (their data pointer is used; dtype and size are
checked here, the library re-checks pointers, alignment and overlap) or as
raw integer device addresses.  ``stream`` defaults to torch's current CUDA
stream.  There is no CPU fallback: if the library is missing, loading fails
with an error.
"""
from __future__ import annotations

import ctypes
import functools
import itertools
import os
import struct
import threading

from . import build as _build

_lock = threading.Lock()
_lib = None

(Z3_OK, Z3_ERR_INVALID_ARG, Z3_ERR_ALIGNMENT, Z3_ERR_OVERFLOW, Z3_ERR_CUDA,
 Z3_ERR_HOST_MEMORY) = range(6)

# Every symbol include/z3.h declares.
EXPORTS = ("z3_layout_create", "z3_layout_destroy", "z3_layout_info", "z3_layout_params",
           "z3_stats", "z3_partition", "z3_allgather", "z3_reduce_scatter",
           "z3_adam_shard_step", "z3_reduce_scatter_adam", "z3_step_layer",
           "z3_allreduce", "z3_scatter", "z3_reshard", "z3_model_step",
           "z3_host_step_create", "z3_host_step_run", "z3_host_step_destroy",
           "z3_step_layer_noalloc", "z3_tensor_list_create", "z3_tensor_list_destroy",
           "z3_grad_norm_workspace_bytes", "z3_grad_norm", "z3_clip",
           "z3_sumsq_len", "z3_reduce_scatter_norm", "z3_adam_shard_step_clipped",
           "z3_model_step_clipped", "z3_head_workspace_bytes", "z3_xent", "z3_xent_grad",
           "z3_distill", "z3_distill_grad", "z3_status_string", "z3_last_error")

# enum z3_dtype
Z3_BF16, Z3_F32, Z3_SUMSQ = range(3)


class Z3Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class AdamHP(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double)]


class Unit(ctypes.Structure):
    """struct z3_unit."""
    _fields_ = [("layout", ctypes.c_void_p), ("shards", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("grads", ctypes.c_void_p), ("grad_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("resident", ctypes.c_void_p),
                ("hp", ctypes.POINTER(AdamHP))]


class Tensor(ctypes.Structure):
    """struct z3_tensor."""
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ClipUnit(ctypes.Structure):
    """struct z3_clip_unit."""
    _fields_ = [("grad_shards", ctypes.c_void_p), ("sumsq", ctypes.c_void_p),
                ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Head(ctypes.Structure):
    """struct z3_head."""
    _fields_ = [("hidden", ctypes.c_void_p), ("hidden_stride", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("weight_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("weights", ctypes.c_void_p)]


class Teacher(ctypes.Structure):
    """struct z3_teacher."""
    _fields_ = [("logits", ctypes.c_void_p), ("index", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("index_bytes", ctypes.c_int32),
                ("k", ctypes.c_int32), ("temperature", ctypes.c_float)]


class Traffic(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "psi", "ag_payload_bytes", "rs_payload_bytes", "step_volume_bytes",
        "dp_allreduce_bytes", "hbm_allgather", "hbm_reduce_scatter",
        "hbm_reduce_scatter_accumulate", "hbm_adam", "hbm_reduce_scatter_adam",
        "hbm_step_layer", "state_bytes_per_rank", "state_bytes_per_rank_fp32_grad")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


def library_path() -> str:
    return _build.LIB_PATH


def load():
    """Load the CUDA library (built by ``optimizer_state_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is not built; run "
                               "`python -m optimizer_state_gb300.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        f32, st = ctypes.c_float, ctypes.c_int
        hp = ctypes.POINTER(AdamHP)
        sig = {
            "z3_layout_create": (st, [vp, i32, i32, ctypes.POINTER(vp)]),
            "z3_layout_destroy": (None, [vp]),
            "z3_layout_info": (st, [vp, vp, vp, vp, vp, vp]),
            "z3_layout_params": (st, [vp, vp, vp, vp, vp]),
            "z3_stats": (st, [vp, ctypes.POINTER(Traffic)]),
            "z3_partition": (st, [vp, vp, vp, vp, vp, vp, vp]),
            "z3_allgather": (st, [vp, vp, vp, vp]),
            "z3_reduce_scatter": (st, [vp, vp, i64, vp, f32, i32, vp]),
            "z3_adam_shard_step": (st, [vp, vp, vp, vp, vp, vp, hp, i64, vp]),
            "z3_reduce_scatter_adam": (st, [vp, vp, i64, f32, vp, vp, vp, vp, vp, hp, i64, vp]),
            "z3_step_layer": (st, [vp, vp, vp, vp, i64, f32, vp, vp, vp, vp, hp, i64, vp]),
            "z3_allreduce": (st, [vp, vp, i64, vp, f32, vp]),
            "z3_scatter": (st, [vp, vp, vp, vp]),
            "z3_reshard": (st, [vp, vp, i32, vp, vp, vp]),
            "z3_model_step": (st, [ctypes.POINTER(Unit), i32, ctypes.POINTER(vp), i32, hp, i64,
                                   vp, vp]),
            "z3_host_step_create": (st, [vp, vp, vp, i64, vp, vp, ctypes.POINTER(vp)]),
            "z3_host_step_run": (st, [vp, vp, vp, vp, f32, vp, vp, vp, hp, i64, vp, vp]),
            "z3_host_step_destroy": (None, [vp]),
            "z3_step_layer_noalloc": (st, [vp, vp, vp, i64, f32, vp, vp, vp, hp, i64, vp]),
            "z3_grad_norm_workspace_bytes": (st, [ctypes.POINTER(i64)]),
            "z3_tensor_list_create": (st, [ctypes.POINTER(Tensor), i32, ctypes.POINTER(vp)]),
            "z3_tensor_list_destroy": (None, [vp]),
            "z3_grad_norm": (st, [vp, f32, vp, vp, vp]),
            "z3_clip": (st, [vp, vp, vp]),
            "z3_sumsq_len": (st, [vp, ctypes.POINTER(i64)]),
            "z3_reduce_scatter_norm": (st, [vp, vp, i64, vp, f32, i32, vp, vp]),
            "z3_adam_shard_step_clipped": (st, [vp, vp, vp, vp, vp, vp, hp, i64, vp, vp]),
            "z3_model_step_clipped": (st, [ctypes.POINTER(Unit), ctypes.POINTER(ClipUnit), i32,
                                           ctypes.POINTER(vp), i32, hp, i64, f32, vp, vp, vp, vp]),
            "z3_head_workspace_bytes": (st, [i64, i64, i64, i32, i32, ctypes.POINTER(i64)]),
            "z3_xent": (st, [ctypes.POINTER(Head), vp, i32, vp, vp, vp, vp, i64, vp]),
            "z3_xent_grad": (st, [ctypes.POINTER(Head), vp, i32, vp, vp, f32, vp, i64, vp, i64, vp,
                                  i64, vp]),
            "z3_distill": (st, [ctypes.POINTER(Head), ctypes.POINTER(Teacher), vp, vp, vp, vp, i64,
                                vp]),
            "z3_distill_grad": (st, [ctypes.POINTER(Head), ctypes.POINTER(Teacher), vp, vp, f32, vp,
                                     i64, vp, i64, vp, i64, vp]),
            "z3_status_string": (ctypes.c_char_p, [st]),
            "z3_last_error": (ctypes.c_size_t, [ctypes.c_char_p, ctypes.c_size_t]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _status_name(status: int) -> str:
    try:
        return load().z3_status_string(status).decode()
    except Exception:  # noqa: BLE001 - only used while formatting an error
        return f"status {status}"


def last_error() -> str:
    lib = load()
    buf = ctypes.create_string_buffer(1024)
    lib.z3_last_error(buf, len(buf))
    return buf.value.decode(errors="replace")


def _check(status: int):
    if status != Z3_OK:
        raise Z3Error(status, last_error())


@functools.cache
def _torch():
    import torch
    return torch


@functools.cache
def _current_device():
    """torch.cuda.current_device without its check that CUDA is up: called
    with a CUDA tensor at hand."""
    return _torch()._C._cuda_getDevice


def _stream(stream):
    if stream is None:
        # the handle alone: torch.cuda.current_stream() builds a stream object
        # around it, which takes as long as a launch
        return _torch()._C._cuda_getCurrentRawStream(_torch().cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dev(t, dtypes, numel: int, name: str):
    """Device address of a tensor (or a raw int address).  A tensor must live
    on the current device: the library launches there, and every kernel
    treats its buffers as that device's own memory."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != _current_device()():
        raise ValueError(f"{name}: on {t.device}, but the current device is "
                         f"cuda:{_torch().cuda.current_device()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs >= {numel} elements, has {t.numel()}")
    return t.data_ptr()


@functools.cache
def _dtypes():
    torch = _torch()
    return (torch.bfloat16, torch.int16, torch.uint16), (torch.float32,)


class Layout:
    """Owns a ``z3_layout`` handle (z3_layout_create / z3_layout_destroy)."""

    def __init__(self, numel, n_ranks: int):
        lib = load()
        numel = [int(n) for n in numel]
        arr = (ctypes.c_int64 * len(numel))(*numel)
        h = ctypes.c_void_p()
        _check(lib.z3_layout_create(ctypes.cast(arr, ctypes.c_void_p), len(numel), n_ranks,
                                    ctypes.byref(h)))
        self._h = h
        self._lib = lib
        P, N = ctypes.c_int32(), ctypes.c_int32()
        S, psi, psip = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib.z3_layout_info(h, ctypes.byref(P), ctypes.byref(N), ctypes.byref(S),
                                  ctypes.byref(psi), ctypes.byref(psip)))
        self.n_params, self.n_ranks = P.value, N.value
        self.S, self.psi, self.psi_padded = S.value, psi.value, psip.value
        arrs = [(ctypes.c_int64 * self.n_params)() for _ in range(4)]
        _check(lib.z3_layout_params(h, *[ctypes.cast(a, ctypes.c_void_p) for a in arrs]))
        self.numel, self.shard_numel, self.shard_off, self.full_off = (list(a) for a in arrs)
        n = ctypes.c_int64()
        _check(lib.z3_sumsq_len(h, ctypes.byref(n)))
        self.sumsq_len = n.value        # doubles of z3_reduce_scatter_norm's sumsq

    @property
    def handle(self):
        return self._h

    def stats(self) -> dict:
        t = Traffic()
        _check(self._lib.z3_stats(self._h, ctypes.byref(t)))
        return t.as_dict()

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.z3_layout_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


def _hp(hp) -> AdamHP:
    if isinstance(hp, AdamHP):
        return hp
    return AdamHP(float(hp["lr"]), float(hp["beta1"]), float(hp["beta2"]), float(hp["eps"]),
                  float(hp.get("weight_decay", 0.0)))


def z3_partition(layout: Layout, full, shards, master, m, v, stream=None):
    b16, f32 = _dtypes()
    T = layout.psi_padded
    _check(load().z3_partition(layout.handle, _dev(full, f32, layout.psi, "full"),
                               _dev(shards, b16, T, "shards"), _dev(master, f32, T, "master"),
                               _dev(m, f32, T, "m"), _dev(v, f32, T, "v"), _stream(stream)))


def z3_allgather(layout: Layout, shards, full, stream=None):
    b16, _ = _dtypes()
    _check(load().z3_allgather(layout.handle, _dev(shards, b16, layout.psi_padded, "shards"),
                               _dev(full, b16, layout.psi, "full"), _stream(stream)))


def z3_reduce_scatter(layout: Layout, grads, grad_stride: int, grad_shards, scale: float,
                      accumulate: bool = False, stream=None):
    b16, f32 = _dtypes()
    _check(load().z3_reduce_scatter(
        layout.handle, _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride,
        _dev(grad_shards, f32, layout.psi_padded, "grad_shards"), scale, 1 if accumulate else 0,
        _stream(stream)))


def z3_adam_shard_step(layout: Layout, master, m, v, grad_shards, shards, hp, step: int,
                       stream=None):
    b16, f32 = _dtypes()
    T = layout.psi_padded
    h = _hp(hp)
    _check(load().z3_adam_shard_step(
        layout.handle, _dev(master, f32, T, "master"), _dev(m, f32, T, "m"),
        _dev(v, f32, T, "v"), _dev(grad_shards, f32, T, "grad_shards"),
        _dev(shards, b16, T, "shards"), ctypes.byref(h), step, _stream(stream)))


def z3_reduce_scatter_adam(layout: Layout, grads, grad_stride: int, scale: float, grad_acc,
                           master, m, v, shards, hp, step: int, stream=None):
    b16, f32 = _dtypes()
    T = layout.psi_padded
    h = _hp(hp)
    _check(load().z3_reduce_scatter_adam(
        layout.handle, _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride,
        scale, _dev(grad_acc, f32, T, "grad_acc"), _dev(master, f32, T, "master"),
        _dev(m, f32, T, "m"), _dev(v, f32, T, "v"), _dev(shards, b16, T, "shards"),
        ctypes.byref(h), step, _stream(stream)))


def z3_step_layer(layout: Layout, shards, full, grads, grad_stride: int, scale: float, master,
                  m, v, hp, step: int, stream=None, grad_shards=None):
    """grad_shards: None (the C call's grad_shards_or_NULL = NULL) or an fp32
    [N*S] tensor that receives the reduced gradient slices."""
    b16, f32 = _dtypes()
    T = layout.psi_padded
    h = _hp(hp)
    _check(load().z3_step_layer(
        layout.handle, _dev(shards, b16, T, "shards"), _dev(full, b16, layout.psi, "full"),
        _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride, scale,
        _dev(master, f32, T, "master"), _dev(m, f32, T, "m"), _dev(v, f32, T, "v"),
        _dev(grad_shards, f32, T, "grad_shards"), ctypes.byref(h), step, _stream(stream)))


def z3_step_layer_noalloc(layout: Layout, shards, grads, grad_stride: int, scale: float, master,
                          m, v, hp, step: int, stream=None):
    """z3_step_layer whose gathers write into the library's own static
    device array instead of a caller buffer: for callers that cannot
    allocate device memory (at most 16,777,216 elements per layer)."""
    b16, f32 = _dtypes()
    T = layout.psi_padded
    h = _hp(hp)
    _check(load().z3_step_layer_noalloc(
        layout.handle, _dev(shards, b16, T, "shards"),
        _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride, scale,
        _dev(master, f32, T, "master"), _dev(m, f32, T, "m"), _dev(v, f32, T, "v"),
        ctypes.byref(h), step, _stream(stream)))


def z3_allreduce(layout: Layout, grads, grad_stride: int, out, scale: float, stream=None):
    b16, f32 = _dtypes()
    _check(load().z3_allreduce(
        layout.handle, _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride,
        _dev(out, f32, layout.psi, "out"), scale, _stream(stream)))


def z3_scatter(layout: Layout, full, shards, stream=None):
    _, f32 = _dtypes()
    _check(load().z3_scatter(layout.handle, _dev(full, f32, layout.psi, "full"),
                             _dev(shards, f32, layout.psi_padded, "shards"), _stream(stream)))


def z3_reshard(src_layout: Layout, dst_layout: Layout, src, dst, stream=None):
    """Element size from the tensors' dtype (bf16: 2 bytes, fp32: 4 bytes)."""
    b16, f32 = _dtypes()
    dt = b16 + f32
    elem = 2 if src.dtype in b16 else 4
    if (dst.dtype in b16) != (elem == 2):
        raise ValueError("src and dst must have the same element size")
    _check(load().z3_reshard(src_layout.handle, dst_layout.handle, elem,
                             _dev(src, dt, src_layout.psi_padded, "src"),
                             _dev(dst, dt, dst_layout.psi_padded, "dst"), _stream(stream)))


def z3_model_step(units, full, hp, step: int, stream=None, gather_stream=None):
    """units: sequence of (layout, shards, master, m, v, grads, grad_stride,
    scale[, resident[, hp]]) -- resident is None for a unit gathered at each
    use, else that unit's persistent bf16 [Psi] copy; hp is None for the
    step's hyperparameters, else this unit's own; full: one transient buffer,
    or D + 1 of them for the prefetching schedule (then gather_stream is
    required)."""
    arr, fulls, _keep = _unit_args(units, full)
    h = _hp(hp)
    _check(load().z3_model_step(arr, len(units), fulls, len(full), ctypes.byref(h), step,
                                _stream(stream),
                                None if gather_stream is None else _stream(gather_stream)))


def _unit_args(units, full):
    """z3_model_step's unit array and transient buffers, and what they point to."""
    b16, f32 = _dtypes()
    arr = (Unit * len(units))()
    own_hp = []                     # kept alive until the call returns
    need = 0
    for i, u in enumerate(units):
        L, sh, ma, m, v, g, stride, scale = u[:8]
        res = u[8] if len(u) > 8 else None
        uhp = u[9] if len(u) > 9 else None
        T = L.psi_padded
        hp_ptr = None
        if uhp is not None:
            own_hp.append(_hp(uhp))
            hp_ptr = ctypes.pointer(own_hp[-1])
        arr[i] = Unit(L.handle.value, _dev(sh, b16, T, "shards"), _dev(ma, f32, T, "master"),
                      _dev(m, f32, T, "m"), _dev(v, f32, T, "v"),
                      _dev(g, b16, L.n_ranks * stride, "grads"), stride, scale,
                      None if res is None else _dev(res, b16, L.psi, "resident"), hp_ptr)
        if res is None:
            need = max(need, L.psi)
    fulls = (ctypes.c_void_p * len(full))(*[_dev(f, b16, need, "full") for f in full])
    return arr, fulls, own_hp


# ---------------------------------------------------------------------------
# gradient clipping by the global norm
# ---------------------------------------------------------------------------

def _records(tensors, kinds, name):
    """The fields of z3_tensor for each tensor, one after the other; kinds: the
    z3_dtype of each dtype allowed."""
    here = _torch().cuda.current_device() if tensors and tensors[0].is_cuda else None
    for i, t in enumerate(tensors):
        kind = kinds.get(t.dtype)
        if kind is None or not t.is_cuda or t.get_device() != here or not t.is_contiguous():
            _dev(t, tuple(kinds), 0, f"{name}[{i}]")    # says what is wrong
        yield t.data_ptr()
        yield t.numel()
        yield kind
        yield 0


class TensorList:
    """Owns a ``z3_tensor_list`` handle (z3_tensor_list_create / _destroy), and
    keeps the tensors alive: bf16 or fp32 CUDA tensors of any lengths
    (contiguous; views into flat buffers may start at any element), and
    `sumsq`, fp64 tensors that z3_reduce_scatter_norm wrote."""

    def __init__(self, tensors, sumsq=()):
        torch = _torch()
        b16, f32 = _dtypes()
        lib = load()
        tensors, sumsq = list(tensors), list(sumsq)
        self._keep = tensors + sumsq
        n = len(self._keep)
        arr = (Tensor * n).from_buffer_copy(struct.pack("Pqii" * n, *itertools.chain(
            _records(tensors, {d: Z3_BF16 for d in b16} | {d: Z3_F32 for d in f32}, "tensors"),
            _records(sumsq, {torch.float64: Z3_SUMSQ}, "sumsq"))))
        h = ctypes.c_void_p()
        _check(lib.z3_tensor_list_create(arr, n, ctypes.byref(h)))
        self._h = h
        self._lib = lib

    def __len__(self):
        return len(self._keep)

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.z3_tensor_list_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


@functools.cache
def _workspace_bytes() -> int:
    n = ctypes.c_int64()
    _check(load().z3_grad_norm_workspace_bytes(ctypes.byref(n)))
    return n.value


def grad_norm_workspace(device=None):
    """A workspace for z3_grad_norm and z3_model_step_clipped."""
    import torch
    return torch.empty(_workspace_bytes(), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def _workspace(t):
    return _dev(t, (_torch().uint8,), _workspace_bytes(), "workspace")


def z3_grad_norm(tensors, max_norm: float, clip, workspace, stream=None):
    """tensors: a TensorList, or a sequence of tensors to make one of; clip:
    fp32 [2], receives {norm, coef}; workspace: grad_norm_workspace()."""
    _, f32 = _dtypes()
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
    _check(load().z3_grad_norm(tensors.handle, max_norm, _dev(clip, f32, 2, "clip"),
                               _workspace(workspace), _stream(stream)))


def z3_clip(tensors, clip, stream=None):
    """Scales the tensors in place by the coef that z3_grad_norm left in clip."""
    _, f32 = _dtypes()
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
    _check(load().z3_clip(tensors.handle, _dev(clip, f32, 2, "clip"), _stream(stream)))


def z3_reduce_scatter_norm(layout: Layout, grads, grad_stride: int, grad_shards, scale: float,
                           sumsq, accumulate: bool = False, stream=None):
    """sumsq: fp64 [layout.sumsq_len], for TensorList(..., sumsq=[...])."""
    import torch
    b16, f32 = _dtypes()
    _check(load().z3_reduce_scatter_norm(
        layout.handle, _dev(grads, b16, layout.n_ranks * grad_stride, "grads"), grad_stride,
        _dev(grad_shards, f32, layout.psi_padded, "grad_shards"), scale, 1 if accumulate else 0,
        _dev(sumsq, (torch.float64,), layout.sumsq_len, "sumsq"), _stream(stream)))


def z3_adam_shard_step_clipped(layout: Layout, master, m, v, grad_shards, shards, hp, step: int,
                               clip, stream=None):
    b16, f32 = _dtypes()
    T = layout.psi_padded
    h = _hp(hp)
    _check(load().z3_adam_shard_step_clipped(
        layout.handle, _dev(master, f32, T, "master"), _dev(m, f32, T, "m"),
        _dev(v, f32, T, "v"), _dev(grad_shards, f32, T, "grad_shards"),
        _dev(shards, b16, T, "shards"), ctypes.byref(h), step, _dev(clip, f32, 2, "clip"),
        _stream(stream)))


def z3_model_step_clipped(units, clips, full, hp, step: int, max_norm: float, clip, workspace,
                          stream=None, gather_stream=None):
    """z3_model_step with the gradients clipped by their global norm.  units,
    full and gather_stream as there; clips: for each unit (grad_shards, sumsq[,
    accumulate]); clip and workspace as for z3_grad_norm."""
    import torch
    _, f32 = _dtypes()
    if len(clips) != len(units):
        raise ValueError(f"clips: {len(clips)} for {len(units)} units")
    arr, fulls, _keep = _unit_args(units, full)
    carr = (ClipUnit * len(units))()
    for i, (u, c) in enumerate(zip(units, clips)):
        L = u[0]
        carr[i] = ClipUnit(_dev(c[0], f32, L.psi_padded, "grad_shards"),
                           _dev(c[1], (torch.float64,), L.sumsq_len, "sumsq"),
                           1 if len(c) > 2 and c[2] else 0, 0)
    h = _hp(hp)
    _check(load().z3_model_step_clipped(
        arr, carr, len(units), fulls, len(full), ctypes.byref(h), step, max_norm,
        _dev(clip, f32, 2, "clip"), _workspace(workspace), _stream(stream),
        None if gather_stream is None else _stream(gather_stream)))


# ---------------------------------------------------------------------------
# losses over a vocabulary
# ---------------------------------------------------------------------------

def head_workspace(tokens: int, dim: int, vocab: int, k: int = 0, grads: bool = True,
                   device=None):
    """A workspace for the calls below at these sizes: k the length of the
    teacher's lists (0: cross entropy), grads for the gradient calls too."""
    import torch
    n = ctypes.c_int64()
    _check(load().z3_head_workspace_bytes(tokens, dim, vocab, k, 1 if grads else 0,
                                          ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device="cuda" if device is None else device)


@functools.cache
def _head_types():
    torch = _torch()
    b16, f32 = _dtypes()
    return b16, f32, (torch.int32, torch.int64), (torch.bfloat16, torch.float32), (torch.uint8,)


def _matrix(t, rows, cols, here, name: str):
    """Address and row stride of a bf16 [rows][cols] CUDA tensor whose rows
    may lie apart."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: needs shape [{rows}, {cols}], has {list(t.shape)}")
    apart, step = t.stride()
    if rows <= 1:
        apart = cols
    if cols > 1 and step != 1 or apart < cols:
        raise ValueError(f"{name}: strides {t.stride()}: rows must be contiguous and apart")
    b16 = _head_types()[0]
    if t.get_device() != here or t.dtype not in b16:
        _dev(t[:0], b16, 0, name)                   # says what is wrong
    return t.data_ptr(), apart


def _vector(t, dtypes, shape, here, name: str):
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name}: needs shape {list(shape)}, has {list(t.shape)}")
    if t.get_device() != here or t.dtype not in dtypes or not t.is_contiguous():
        _dev(t, dtypes, 0, name)                    # says what is wrong
    return t.data_ptr()


class _HeadCall:
    """The arguments that the calls below share, from tensors."""

    def __init__(self, hidden, weight, weights, workspace, stream):
        if hidden.dim() != 2 or weight.dim() != 2:
            t, name = (weight, "weight") if hidden.dim() == 2 else (hidden, "hidden")
            raise ValueError(f"{name}: needs two dimensions, has shape {list(t.shape)}")
        self.n, self.d = n, d = hidden.shape
        self.v = v = weight.shape[0]
        self.here = here = _current_device()() if hidden.is_cuda else None
        h, hs = _matrix(hidden, n, d, here, "hidden")
        w, ws = _matrix(weight, v, d, here, "weight")
        self.head = ctypes.byref(Head(h, hs, w, ws, n, v, d, self.vector(weights, 1, (n,),
                                                                         "weights")))
        space = workspace.numel()
        if stream is None:
            stream = _torch()._C._cuda_getCurrentRawStream(here)
        self.end = (_vector(workspace, _head_types()[4], (space,), here, "workspace"), space,
                    _stream(stream))

    def vector(self, t, kind, shape, name):
        return _vector(t, _head_types()[kind], shape, self.here, name)

    def targets(self, t):
        return self.vector(t, 2, (self.n,), "targets"), t.element_size()

    def teacher(self, t, index, temperature):
        if t.dim() != 2:
            raise ValueError(f"teacher: needs two dimensions, has shape {list(t.shape)}")
        k = t.shape[1]
        return ctypes.byref(Teacher(
            self.vector(t, 3, (self.n, k), "teacher"), self.vector(index, 2, (self.n, k), "index"),
            Z3_F32 if t.element_size() == 4 else Z3_BF16, index.element_size(), k, temperature))

    def losses(self, loss, lse, total):
        n = (self.n,)
        return (self.vector(loss, 1, n, "loss"), self.vector(lse, 1, n, "lse"),
                self.vector(total, 1, (2,), "total"))

    def grads(self, lse, total, scale, d_hidden, d_weight):
        return (self.vector(lse, 1, (self.n,), "lse"), self.vector(total, 1, (2,), "total"), scale,
                *_matrix(d_hidden, self.n, self.d, self.here, "d_hidden"),
                *_matrix(d_weight, self.v, self.d, self.here, "d_weight"))


def z3_xent(hidden, weight, targets, loss, lse, total, workspace, weights=None, stream=None):
    """Softmax cross entropy of hidden [tokens, dim] against the vocabulary of
    weight [vocab, dim] (bf16; rows may lie apart), without its logits.
    targets: int32 or int64 [tokens], negative ones left out; weights: fp32
    [tokens] or None; loss and lse: fp32 [tokens], total: fp32 [2], receive the
    tokens' losses and {sum of weighted losses, sum of weights}."""
    c = _HeadCall(hidden, weight, weights, workspace, stream)
    _check(load().z3_xent(c.head, *c.targets(targets), *c.losses(loss, lse, total), *c.end))


def z3_xent_grad(hidden, weight, targets, lse, total, scale: float, d_hidden, d_weight, workspace,
                 weights=None, stream=None):
    """The gradients of scale * total[0] / total[1] (total None: of scale times
    the sum) into d_hidden and d_weight, either of which may be None; lse and
    total as z3_xent wrote them."""
    c = _HeadCall(hidden, weight, weights, workspace, stream)
    _check(load().z3_xent_grad(c.head, *c.targets(targets),
                               *c.grads(lse, total, scale, d_hidden, d_weight), *c.end))


def z3_distill(hidden, weight, teacher, index, temperature: float, loss, lse, total, workspace,
               weights=None, stream=None):
    """Divergence of the head's softmax from that of a teacher's k highest
    logits, teacher [tokens, k] (bf16 or fp32) at the words index [tokens, k]
    (int32 or int64; negative ones left out).  The rest as z3_xent."""
    c = _HeadCall(hidden, weight, weights, workspace, stream)
    _check(load().z3_distill(c.head, c.teacher(teacher, index, temperature),
                             *c.losses(loss, lse, total), *c.end))


def z3_distill_grad(hidden, weight, teacher, index, temperature: float, lse, total, scale: float,
                    d_hidden, d_weight, workspace, weights=None, stream=None):
    c = _HeadCall(hidden, weight, weights, workspace, stream)
    _check(load().z3_distill_grad(c.head, c.teacher(teacher, index, temperature),
                                  *c.grads(lse, total, scale, d_hidden, d_weight), *c.end))


def _host(t, dtypes, numel: int, name: str):
    """Host address of a CPU tensor (or a raw int address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.is_cuda:
        raise ValueError(f"{name}: must be a host (CPU) tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs >= {numel} elements, has {t.numel()}")
    return t.data_ptr()


class HostStep:
    """z3_host_step_create / _run / _destroy: the layer step fed from host
    memory through two device staging buffers (caller-owned tensors kept
    alive by this object)."""

    def __init__(self, layout: Layout, staging0, staging1, grad_stride: int, upload_stream,
                 download_stream):
        b16, _ = _dtypes()
        n = layout.n_ranks * grad_stride
        self._keep = (layout, staging0, staging1, upload_stream, download_stream)
        self.layout, self.grad_stride = layout, grad_stride
        h = ctypes.c_void_p()
        _check(load().z3_host_step_create(
            layout.handle, _dev(staging0, b16, n, "staging0"), _dev(staging1, b16, n, "staging1"),
            grad_stride, _stream(upload_stream), _stream(download_stream), ctypes.byref(h)))
        self._h = h

    def run(self, grads_host, shards, full, scale: float, master, m, v, hp, step: int,
            shards_host=None, stream=None):
        b16, f32 = _dtypes()
        L = self.layout
        T = L.psi_padded
        h = _hp(hp)
        _check(load().z3_host_step_run(
            self._h, _host(grads_host, b16, L.n_ranks * self.grad_stride, "grads_host"),
            _dev(shards, b16, T, "shards"), _dev(full, b16, L.psi, "full"), scale,
            _dev(master, f32, T, "master"), _dev(m, f32, T, "m"), _dev(v, f32, T, "v"),
            ctypes.byref(h), step, _host(shards_host, b16, T, "shards_host"), _stream(stream)))

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            load().z3_host_step_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass
