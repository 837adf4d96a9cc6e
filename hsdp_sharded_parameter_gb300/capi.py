"""Thin Python binding of the C-ABI library (include/hsdp_fsdp.h).

Argument marshalling only: every step of the data path runs in the
library's CUDA kernels. Functions keep the C names; ``Plan`` and
``Binding`` own the C handles. Tensors are passed as device pointers
(``data_ptr()``); streams as ``torch.cuda.Stream`` or raw handles.

The library must have been built (``python -m hsdp_sharded_parameter_gb300.build``
or ``__graft_entry__.build()``): there is no fallback of any kind, a missing
library raises.
"""
from __future__ import annotations

import ctypes
import os
import re

from .build import library_path

FSDP_OK, FSDP_ERR_INVALID_ARG, FSDP_ERR_NOT_IMPLEMENTED, FSDP_ERR_CUDA, FSDP_ERR_NOMEM = range(5)
FSDP_F32, FSDP_BF16 = 0, 1
FSDP_AVG, FSDP_SUM = 0, 1
FSDP_I32, FSDP_I64 = 0, 1
FSDP_SILU, FSDP_GELU, FSDP_RELU = 0, 1, 2
FSDP_STATUS_PRODUCER_WAIT, FSDP_STATUS_CONSUMER_WAIT, FSDP_STATUS_ORDER = 1, 2, 4
(FSDP_ROLE_SHARDS, FSDP_ROLE_AG_OUTPUT, FSDP_ROLE_FULL_PARAMS, FSDP_ROLE_GRADS,
 FSDP_ROLE_RS_INPUT, FSDP_ROLE_FUSED, FSDP_ROLE_SHARD_GRADS) = range(7)

ROLES = {"shards": FSDP_ROLE_SHARDS, "ag_output": FSDP_ROLE_AG_OUTPUT,
         "full_params": FSDP_ROLE_FULL_PARAMS, "grads": FSDP_ROLE_GRADS,
         "rs_input": FSDP_ROLE_RS_INPUT, "fused": FSDP_ROLE_FUSED,
         "shard_grads": FSDP_ROLE_SHARD_GRADS}
DTYPES = {"f32": FSDP_F32, "bf16": FSDP_BF16}
# roles that take one buffer per (rank, parameter); the others one per rank
PER_PARAM_ROLES = {FSDP_ROLE_SHARDS, FSDP_ROLE_FULL_PARAMS, FSDP_ROLE_GRADS, FSDP_ROLE_SHARD_GRADS}
OPS = {"avg": FSDP_AVG, "sum": FSDP_SUM}
ACTIVATIONS = {"silu": FSDP_SILU, "gelu": FSDP_GELU, "relu": FSDP_RELU}

_lib = None


class FsdpError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"[status {code}] {msg}")
        self.code = code


def header_symbols():
    """Names of the functions include/hsdp_fsdp.h declares."""
    hdr = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                       "hsdp_fsdp.h")
    text = open(hdr).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fsdp_[a-z0-9_]+)\s*\(", text)))


def lib():
    """The loaded C-ABI library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library not built: {path} is missing "
                               "(run __graft_entry__.build())")
        L = ctypes.CDLL(path)
        i32, i64, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
        P = ctypes.POINTER
        L.fsdp_last_error.restype = ctypes.c_char_p
        L.fsdp_launch_count.restype = ctypes.c_uint64
        L.fsdp_plan_create.argtypes = [i32, vp, vp, i32, i32, i32, i32, P(vp)]
        L.fsdp_plan_create_bucketed.argtypes = [i32, vp, vp, vp, i32, i32, i32, i32, P(vp)]
        L.fsdp_plan_destroy.argtypes = [vp]
        L.fsdp_plan_upload.argtypes = [vp]
        L.fsdp_plan_set_grid_limit.argtypes = [vp, i32]
        L.fsdp_plan_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
        L.fsdp_plan_inject_stall.argtypes = [vp, i32]
        L.fsdp_plan_status.argtypes = [vp, vp, P(i32)]
        L.fsdp_plan_check_tables.argtypes = [vp]
        L.fsdp_plan_info.argtypes = [vp, P(i32), P(i32), P(i32), P(i32), P(i64)]
        L.fsdp_slice_numel.argtypes = [vp, i32, P(i64)]
        L.fsdp_sharded_size.argtypes = [vp, i32, i32, P(i64), P(i64)]
        L.fsdp_padded_sharded_param_size.argtypes = [vp, i32, P(i64)]
        L.fsdp_offsets.argtypes = [vp, vp]
        L.fsdp_group_ranks.argtypes = [vp, i32, vp, vp]
        L.fsdp_comm_calls.argtypes = [vp, P(i32), P(i32)]
        L.fsdp_bind.argtypes = [vp, i32, i32, vp, vp, P(vp)]
        L.fsdp_binding_destroy.argtypes = [vp]
        L.fsdp_ag_copy_in.argtypes = [vp, vp, vp, i32, vp]
        L.fsdp_ag_gather.argtypes = [vp, vp, vp]
        L.fsdp_ag_copy_out.argtypes = [vp, vp, vp, vp]
        L.fsdp_rs_copy_in.argtypes = [vp, vp, vp, vp]
        L.fsdp_rs_ar_reduce.argtypes = [vp, vp, vp, vp]
        L.fsdp_apply_grads.argtypes = [vp, vp, i32, i32, vp, vp]
        L.fsdp_rs_reduce.argtypes = [vp, vp, i32, vp, vp]
        L.fsdp_rs_ar_reduce_apply.argtypes = [vp, vp, vp, i32, i32, vp, vp]
        L.fsdp_ar_reduce.argtypes = [vp, vp, i32, vp]
        L.fsdp_rs_ar_reduce_noalloc.argtypes = [vp, i32, vp, vp, vp]
        L.fsdp_ag_unshard.argtypes = [vp, vp, vp, vp]
        f64, u32, u64, sz = ctypes.c_double, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t
        L.fsdp_embedding.argtypes = [i32, vp, i64, i64, i64, i32, vp, i64, i64, f64, i32, vp, i64, vp]
        L.fsdp_embedding_grad_workspace.argtypes = [i64, i64, i64, P(sz)]
        L.fsdp_embedding_grad.argtypes = [i32, vp, i64, i32, vp, i64, i64, f64, i32, i32, vp, i64, i64, i64, vp, sz, vp]
        L.fsdp_dropout.argtypes = [i64, i64, i32, vp, i64, vp, i64, f64, u64, u32, vp, i64, vp]
        L.fsdp_layer_norm.argtypes = [i64, i64, i32, vp, i64, vp, i64, f64, u64, u32, i32, vp, vp, f64, vp, i64, vp,
                                      i64, vp, vp, vp]
        L.fsdp_layer_norm_grad_workspace.argtypes = [i64, i64, P(sz)]
        L.fsdp_layer_norm_grad.argtypes = [i64, i64, i32, vp, i64, vp, i64, vp, i64, vp, vp, i32, vp, f64, u64, u32,
                                           i32, vp, i64, vp, i64, i32, vp, vp, vp, sz, vp]
        L.fsdp_operators_status.argtypes = [vp, P(i32)]
        L.fsdp_gated_ffn_workspace.argtypes = [i64, i64, i64, i32, P(sz)]
        L.fsdp_gated_ffn.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64, vp, i64,
                                     vp, sz, vp]
        L.fsdp_gated_ffn_grad_workspace.argtypes = [i64, i64, i64, i32, P(sz)]
        L.fsdp_gated_ffn_grad.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                          i32, vp, i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, sz, vp]
        L.fsdp_orthogonalize_workspace.argtypes = [i64, i64, P(sz)]
        L.fsdp_orthogonalize.argtypes = [i64, i64, i32, vp, i64, i32, f64, f64, f64, f64, f64, vp, i64, vp, sz, vp]
        _lib = L
    return _lib


def _check(code):
    if code != FSDP_OK:
        raise FsdpError(code, lib().fsdp_last_error().decode())


def _stream(stream):
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream
        except Exception:
            return 0
    return getattr(stream, "cuda_stream", stream)


def fsdp_launch_count():
    return int(lib().fsdp_launch_count())


class Plan:
    """Owns an fsdp_plan_t. Host-only until ``upload()``."""

    def __init__(self, dim0, inner, rank_size, shard_size, enable_param_shard=1, shard_dim=0,
                 bucket=None):
        import numpy as np

        self._d0 = np.ascontiguousarray(dim0, dtype=np.int64)
        self._inner = np.ascontiguousarray(inner, dtype=np.int64)
        self._bucket = None if bucket is None else np.ascontiguousarray(bucket, dtype=np.int32)
        h = ctypes.c_void_p()
        _check(lib().fsdp_plan_create_bucketed(
            len(self._d0), self._d0.ctypes.data, self._inner.ctypes.data,
            None if self._bucket is None else self._bucket.ctypes.data,
            rank_size, shard_size, enable_param_shard, shard_dim, ctypes.byref(h)))
        self.handle = h
        W, S, D, P = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        sp = ctypes.c_int64()
        _check(lib().fsdp_plan_info(h, ctypes.byref(W), ctypes.byref(S), ctypes.byref(D),
                                    ctypes.byref(P), ctypes.byref(sp)))
        self.W, self.S, self.D, self.P, self.sum_padded = W.value, S.value, D.value, P.value, sp.value

    def close(self):
        if getattr(self, "handle", None):
            lib().fsdp_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def upload(self):
        _check(lib().fsdp_plan_upload(self.handle))
        return self

    def check_tables(self):
        """Host-side bounds and coverage check of the plan's work tables
        (no GPU needed); raises FsdpError naming the first violation."""
        _check(lib().fsdp_plan_check_tables(self.handle))
        return self

    def set_grid_limit(self, max_blocks):
        _check(lib().fsdp_plan_set_grid_limit(self.handle, int(max_blocks)))
        return self

    def set_wait_limit(self, nanoseconds):
        _check(lib().fsdp_plan_set_wait_limit(self.handle, int(nanoseconds)))
        return self

    def inject_stall(self, on=True):
        _check(lib().fsdp_plan_inject_stall(self.handle, int(bool(on))))
        return self

    def status(self, stream=None):
        """The plan's status word after the calls enqueued on `stream` (the
        stream is synchronised; the word is cleared): 0, or the
        FSDP_STATUS_* bits of waits that ran out."""
        v = ctypes.c_int(0)
        _check(lib().fsdp_plan_status(self.handle, _stream(stream), ctypes.byref(v)))
        return v.value

    def slice_numel(self, dt):
        out = ctypes.c_int64()
        _check(lib().fsdp_slice_numel(self.handle, DTYPES.get(dt, dt), ctypes.byref(out)))
        return out.value

    def sharded_size(self, p, s):
        a, n = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().fsdp_sharded_size(self.handle, p, s, ctypes.byref(a), ctypes.byref(n)))
        return a.value, n.value

    def padded_sharded_param_size(self, p):
        c = ctypes.c_int64()
        _check(lib().fsdp_padded_sharded_param_size(self.handle, p, ctypes.byref(c)))
        return c.value

    def offsets(self):
        import numpy as np

        o = np.zeros(self.P + 1, np.int64)
        _check(lib().fsdp_offsets(self.handle, o.ctypes.data))
        return o

    def group_ranks(self, w):
        import numpy as np

        sg = np.zeros(self.S, np.int32)
        rg = np.zeros(self.D, np.int32)
        _check(lib().fsdp_group_ranks(self.handle, w, sg.ctypes.data, rg.ctypes.data))
        return sg, rg

    def comm_calls(self):
        rs, ar = ctypes.c_int(), ctypes.c_int()
        _check(lib().fsdp_comm_calls(self.handle, ctypes.byref(rs), ctypes.byref(ar)))
        return rs.value, ar.value

    # sizes the caller allocates
    def shard_numel(self, p, s):
        _, n = self.sharded_size(p, s)
        return n * int(self._inner[p])

    def numel(self, p):
        return int(self._d0[p] * self._inner[p])

    def bind(self, role, dt, tensors, check_sizes=True):
        return Binding(self, role, dt, tensors, check_sizes)


def _torch_dtype(dt):
    import torch

    return {FSDP_F32: torch.float32, FSDP_BF16: torch.bfloat16}.get(DTYPES.get(dt, dt))


def _check_tensors(what, tensors, count, dt, numel_of=None):
    """Host-side checks before a pointer array goes to the library, which
    reads exactly `count` entries: the count, then (when dt is given) each
    tensor's dtype, device and contiguity, and (numel_of(i)) its size."""
    if len(tensors) != count:
        raise FsdpError(FSDP_ERR_INVALID_ARG, f"{what}: {len(tensors)} tensors given, the plan needs {count}")
    if dt is None:
        return
    want = _torch_dtype(dt)
    for i, t in enumerate(tensors):
        if t.dtype != want or not t.is_cuda or not t.is_contiguous():
            raise FsdpError(FSDP_ERR_INVALID_ARG,
                            f"{what}: tensor {i} is {t.dtype} on {t.device}"
                            f"{'' if t.is_contiguous() else ', not contiguous'}; expected contiguous {want} on a GPU")
        if numel_of is not None and t.numel() < numel_of(i):
            raise FsdpError(FSDP_ERR_INVALID_ARG,
                            f"{what}: tensor {i} holds {t.numel()} elements, needs {numel_of(i)}")


class Binding:
    """Owns an fsdp_binding_t: a device table of the tensors' pointers.
    Keeps the tensors alive while the binding lives. The number of tensors
    is always checked (the library reads W*P or W pointers); with
    check_sizes (the default) their dtypes and sizes are checked too, the
    sizes again by the library."""

    def __init__(self, plan, role, dt, tensors, check_sizes=True):
        r = ROLES.get(role, role)
        _check_tensors(f"bind {role}", tensors, plan.W * plan.P if r in PER_PARAM_ROLES else plan.W,
                       dt if check_sizes else None)
        n = len(tensors)
        ptrs = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in tensors])
        numels = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in tensors])
        h = ctypes.c_void_p()
        _check(lib().fsdp_bind(plan.handle, ROLES.get(role, role), DTYPES.get(dt, dt), ptrs,
                               numels if check_sizes else None, ctypes.byref(h)))
        self.handle = h
        self.plan = plan
        self.tensors = list(tensors)

    def close(self):
        if getattr(self, "handle", None):
            lib().fsdp_binding_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fsdp_ag_copy_in(plan, shards, ag_out, fuse_gather=False, stream=None):
    _check(lib().fsdp_ag_copy_in(plan.handle, shards.handle, ag_out.handle, int(bool(fuse_gather)),
                                 _stream(stream)))


def fsdp_ag_gather(plan, ag_out, stream=None):
    _check(lib().fsdp_ag_gather(plan.handle, ag_out.handle, _stream(stream)))


def fsdp_ag_copy_out(plan, ag_out, full_params, stream=None):
    _check(lib().fsdp_ag_copy_out(plan.handle, ag_out.handle, full_params.handle, _stream(stream)))


def fsdp_ag_unshard(plan, shards, full_params, stream=None):
    _check(lib().fsdp_ag_unshard(plan.handle, shards.handle, full_params.handle, _stream(stream)))


def fsdp_rs_copy_in(plan, grads, rs_in, stream=None):
    _check(lib().fsdp_rs_copy_in(plan.handle, grads.handle, rs_in.handle, _stream(stream)))


def fsdp_rs_ar_reduce(plan, grads, fused, stream=None):
    _check(lib().fsdp_rs_ar_reduce(plan.handle, grads.handle, fused.handle, _stream(stream)))


def fsdp_apply_grads(plan, fused, op, shard_grads, accumulate=False, stream=None):
    _check(lib().fsdp_apply_grads(plan.handle, fused.handle, OPS.get(op, op), int(bool(accumulate)),
                                  shard_grads.handle, _stream(stream)))


def fsdp_rs_ar_reduce_apply(plan, grads, fused, op, shard_grads, accumulate=False, stream=None):
    _check(lib().fsdp_rs_ar_reduce_apply(plan.handle, grads.handle, fused.handle, OPS.get(op, op),
                                         int(bool(accumulate)), shard_grads.handle, _stream(stream)))


def fsdp_rs_reduce(plan, rs_in, op, fused, stream=None):
    _check(lib().fsdp_rs_reduce(plan.handle, rs_in.handle, OPS.get(op, op), fused.handle,
                                _stream(stream)))


def fsdp_ar_reduce(plan, fused, op, stream=None):
    _check(lib().fsdp_ar_reduce(plan.handle, fused.handle, OPS.get(op, op), _stream(stream)))


def fsdp_rs_ar_reduce_noalloc(plan, grad_dt, grads, fused, stream=None):
    """The fused gradient sync without any device allocation by the library
    (for callers that cannot allocate device memory): ``plan`` needs no
    upload, ``grads`` (W*P tensors) and ``fused`` (W fp32 tensors) are passed
    as pointer arrays on every call. The library cannot see the tensors'
    sizes here, so their count, dtype and size are checked before the call."""
    P = plan.P
    # both counts first (the library reads both arrays), then each tensor
    _check_tensors("rs_ar_reduce_noalloc grads", grads, plan.W * P, None)
    _check_tensors("rs_ar_reduce_noalloc fused", fused, plan.W, None)
    _check_tensors("rs_ar_reduce_noalloc grads", grads, plan.W * P, grad_dt, lambda i: plan.numel(i % P))
    sf = plan.slice_numel("f32")
    _check_tensors("rs_ar_reduce_noalloc fused", fused, plan.W, "f32", lambda i: sf)
    g = (ctypes.c_void_p * max(len(grads), 1))(*[t.data_ptr() for t in grads])
    f = (ctypes.c_void_p * max(len(fused), 1))(*[t.data_ptr() for t in fused])
    _check(lib().fsdp_rs_ar_reduce_noalloc(plan.handle, DTYPES.get(grad_dt, grad_dt), g, f,
                                           _stream(stream)))


# --------------------------------------------------------- training operators
#
# Tensors are passed as they are: matrices of 2 dimensions with any row
# stride and neighbouring columns, or contiguous tensors of any other number
# of dimensions, the last being the columns. Outputs and workspaces are the
# caller's. Operators run on the current device and, by default, its current
# stream; on another stream the caller orders the tensors' other uses.

_TYPES = {}


def _types():
    """torch dtypes of the operators' values and of their ids, as the C ABI's.
    The table appears whole: other threads may be at their first call too."""
    global _TYPES
    import torch

    _TYPES = {
        torch.float32: FSDP_F32, torch.bfloat16: FSDP_BF16,
        "ids": {torch.int32: FSDP_I32, torch.int64: FSDP_I64},
        "device": torch.cuda.current_device,
        # the current stream's handle without a Stream object around it (2.8 us a call)
        "stream": getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream),
    }
    return _TYPES


def _refuse(what, why):
    raise FsdpError(FSDP_ERR_INVALID_ARG, f"{what}: {why}")


def _matrix(what, name, t):
    """(pointer, rows, columns, row stride, dtype, device) of a tensor."""
    shape, strides = t.shape, t.stride()
    n = len(shape)
    dt = (_TYPES or _types()).get(t.dtype)
    if dt is None or not t.is_cuda:
        _refuse(what, f"{name} is {t.dtype} on {t.device}; expected float32 or bfloat16 on a GPU")
    if n == 2:
        rows, cols = shape
        stride = strides[0]
        if strides[1] != 1 and cols > 1:
            _refuse(what, f"{name}'s columns are not neighbours in memory (strides {tuple(strides)})")
    else:
        if n == 0 or not t.is_contiguous():
            _refuse(what, f"{name} is neither a matrix nor contiguous")
        cols = stride = shape[-1]
        rows = t.numel() // cols if cols else 0
    return t.data_ptr(), rows, cols, stride, dt, t.get_device()


def _like(what, name, t, rows, cols, dt, dev):
    """Pointer and row stride of a tensor that has to match these, (None, 0) of None."""
    if t is None:
        return None, 0
    p, r, c, stride, d, v = _matrix(what, name, t)
    if r != rows or c != cols or (d != dt and dt is not None) or v != dev:
        _refuse(what, f"{name} is {r} x {c} {t.dtype} on {t.device}; expected {rows} x {cols} "
                      f"{_torch_dtype(dt) if dt is not None else ''} on cuda:{dev}")
    return p, stride


def _on(what, dev, stream):
    """The stream's handle; the tensors' device has to be the current one."""
    if dev != _TYPES["device"]():
        _refuse(what, f"the tensors are on cuda:{dev}, which is not the current device")
    return _TYPES["stream"](dev) if stream is None else getattr(stream, "cuda_stream", stream)


def _vector(what, name, t, n, dev, dtype=None):
    """(pointer, dtype) of a contiguous vector of n values, (None, None) of None."""
    if t is None:
        return None, None
    dt = _TYPES.get(t.dtype)
    if dt is None or (dtype is not None and dt != dtype) or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        _refuse(what, f"{name} is {tuple(t.shape)} {t.dtype} on {t.device}; expected {n} contiguous values of "
                      f"{'float32 or bfloat16' if dtype is None else _torch_dtype(dtype)} on cuda:{dev}")
    return t.data_ptr(), dt


def _pair(what, names, a, b, n, dev):
    """Pointers and the common dtype of two optional parameter vectors."""
    pa, da = _vector(what, names[0], a, n, dev)
    pb, db = _vector(what, names[1], b, n, dev, da)
    return pa, pb, da if da is not None else (db if db is not None else FSDP_F32)


def _ids(what, ids, dev):
    t = _TYPES["ids"].get(ids.dtype)
    if t is None or not ids.is_contiguous() or ids.get_device() != dev:
        _refuse(what, f"ids is {ids.dtype} on {ids.device}; expected contiguous int32 or int64 on cuda:{dev}")
    return t, ids.data_ptr(), ids.numel()


def _work(what, t, dev):
    if not t.is_contiguous() or t.get_device() != dev:
        _refuse(what, f"workspace is not a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


# Numbers that do not fit the C ABI's types would be cut: another first row, or
# the mask of another draw again. (Negative draws and seeds stand for their
# bits.) Compared in the calls themselves, which a function would cost 0.1 us.
_I32, _I64 = -(1 << 31), -(1 << 63)
_U32, _U64, _TOP64 = (1 << 32) - 1, (1 << 64) - 1, (1 << 63) - 1


def _no_mask(what, seed, draw):
    _refuse(what, f"seed {seed} does not fit 64 bits" if _I32 <= draw <= _U32 else f"draw {draw} does not fit 32 bits")


def _no_row(what, first_row):
    _refuse(what, f"first_row {first_row} does not fit 64 bits")


def fsdp_embedding(table, ids, out, scale=1.0, first_row=0, stream=None):
    """out[t] = scale * table[ids[t] - first_row], zeros where the id names no
    row of the table. table: (vocab, cols); ids: n int32 or int64; out:
    (n, cols), float32 or bfloat16 whatever the table's type."""
    what = "embedding"
    if not _I64 <= first_row <= _TOP64:
        _no_row(what, first_row)
    tp, vocab, cols, ts, tdt, dev = _matrix(what, "table", table)
    it, ip, n = _ids(what, ids, dev)
    op, rows, ocols, os_, odt, odev = _matrix(what, "out", out)
    if n and (rows != n or ocols != cols) or odev != dev:
        _refuse(what, f"out is {rows} x {ocols} on cuda:{odev}; expected {n} x {cols} on cuda:{dev}")
    handle = _on(what, dev, stream)
    _check(lib().fsdp_embedding(tdt, tp, ts, vocab, cols, it, ip, n, first_row, scale, odt, op, os_, handle))


def fsdp_embedding_grad_workspace(n_ids, vocab, cols):
    """Bytes of the workspace that fsdp_embedding_grad needs for n_ids tokens or fewer, into vocab rows or fewer."""
    b = ctypes.c_size_t()
    _check(lib().fsdp_embedding_grad_workspace(n_ids, vocab, cols, ctypes.byref(b)))
    return b.value


def fsdp_embedding_grad(grad_out, ids, grad_table, workspace, scale=1.0, first_row=0, accumulate=False, stream=None):
    """grad_table[v] = scale * sum of grad_out[t] over the tokens t that name
    row v, in an order that is the same for equal calls; zeros where there is
    none. With accumulate, added to what grad_table holds. workspace: a tensor
    of at least fsdp_embedding_grad_workspace(n, vocab, cols) bytes."""
    what = "embedding_grad"
    if not _I64 <= first_row <= _TOP64:
        _no_row(what, first_row)
    gp, rows, cols, gs, gdt, dev = _matrix(what, "grad_out", grad_out)
    it, ip, n = _ids(what, ids, dev)
    tp, vocab, tcols, ts, tdt, tdev = _matrix(what, "grad_table", grad_table)
    if n and (rows != n or cols != tcols) or tdev != dev:
        _refuse(what, f"grad_out is {rows} x {cols}, ids {n}, grad_table {vocab} x {tcols} on cuda:{tdev}")
    wp, wb = _work(what, workspace, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_embedding_grad(gdt, gp, gs, it, ip, n, first_row, scale, int(accumulate), tdt, tp, ts, vocab,
                                     tcols, wp, wb, handle))


def fsdp_dropout(x, out, p, seed, draw=0, residual=None, stream=None):
    """out = residual + dropout(x): an element of row r and column c is kept,
    and scaled, by a mask that (seed, draw, r, c) give and nothing stores. The
    backward pass is this call on the gradient. out may be x or residual. seed
    has 64 bits, draw 32."""
    what = "dropout"
    if not (_I32 <= draw <= _U32 and _I64 <= seed <= _U64):
        _no_mask(what, seed, draw)
    xp, rows, cols, xs, dt, dev = _matrix(what, "x", x)
    rp, rs = _like(what, "residual", residual, rows, cols, dt, dev)
    op, os_ = _like(what, "out", out, rows, cols, dt, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_dropout(rows, cols, dt, xp, xs, rp, rs, p, seed, draw, op, os_, handle))


def fsdp_layer_norm(x, weight, bias, out, mean, rstd, eps=1e-5, residual=None, hidden=None, p=0.0, seed=0, draw=0,
                    stream=None):
    """out = layer norm of the rows of h = residual + dropout(x) (no residual,
    p = 0: of x), times weight plus bias (either may be None). hidden receives
    h, mean and rstd (float32) each row's; any of the three may be None."""
    what = "layer_norm"
    if not (_I32 <= draw <= _U32 and _I64 <= seed <= _U64):
        _no_mask(what, seed, draw)
    xp, rows, cols, xs, dt, dev = _matrix(what, "x", x)
    rp, rs = _like(what, "residual", residual, rows, cols, dt, dev)
    hp, hs = _like(what, "hidden", hidden, rows, cols, dt, dev)
    op, os_ = _like(what, "out", out, rows, cols, dt, dev)
    wp, bp, pdt = _pair(what, ("weight", "bias"), weight, bias, cols, dev)
    mp, _ = _vector(what, "mean", mean, rows, dev, FSDP_F32)
    sp, _ = _vector(what, "rstd", rstd, rows, dev, FSDP_F32)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_layer_norm(rows, cols, dt, xp, xs, rp, rs, p, seed, draw, pdt, wp, bp, eps, hp, hs, op, os_, mp,
                                 sp, handle))


def fsdp_layer_norm_grad_workspace(rows, cols):
    """Bytes of the workspace that fsdp_layer_norm_grad needs for that many rows or fewer."""
    b = ctypes.c_size_t()
    _check(lib().fsdp_layer_norm_grad_workspace(rows, cols, ctypes.byref(b)))
    return b.value


def fsdp_layer_norm_grad(grad_out, hidden, mean, rstd, weight, grad_x, grad_weight, grad_bias, workspace,
                         grad_hidden=None, grad_residual=None, p=0.0, seed=0, draw=0, accumulate=False, stream=None):
    """Gradient of fsdp_layer_norm from its hidden (x where it had neither
    residual nor dropout), mean and rstd: grad_x, grad_residual (the same
    before the dropout; may be None), grad_weight and grad_bias (either may be
    None; with accumulate, added to what they hold). grad_hidden is the
    gradient that reaches hidden past the norm. workspace: a tensor of at least
    fsdp_layer_norm_grad_workspace(rows, cols) bytes."""
    what = "layer_norm_grad"
    if not (_I32 <= draw <= _U32 and _I64 <= seed <= _U64):
        _no_mask(what, seed, draw)
    gp, rows, cols, gs, dt, dev = _matrix(what, "grad_out", grad_out)
    hp, hs = _like(what, "hidden", hidden, rows, cols, dt, dev)
    ap, as_ = _like(what, "grad_hidden", grad_hidden, rows, cols, dt, dev)
    rp, rs = _like(what, "grad_residual", grad_residual, rows, cols, dt, dev)
    xp, xs = _like(what, "grad_x", grad_x, rows, cols, dt, dev)
    mp, _ = _vector(what, "mean", mean, rows, dev, FSDP_F32)
    sp, _ = _vector(what, "rstd", rstd, rows, dev, FSDP_F32)
    wp, wdt = _vector(what, "weight", weight, cols, dev)
    dwp, dbp, gdt = _pair(what, ("grad_weight", "grad_bias"), grad_weight, grad_bias, cols, dev)
    kp, kb = _work(what, workspace, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_layer_norm_grad(rows, cols, dt, gp, gs, ap, as_, hp, hs, mp, sp, FSDP_F32 if wdt is None else wdt,
                                      wp, p, seed, draw, int(accumulate), rp, rs, xp, xs, gdt, dwp, dbp, kp, kb,
                                      handle))


# ----------------------------------------- products of a feed-forward block
#
# Matrices are passed as above, in bfloat16 where nothing else is said. A sum has
# up to 2^24 terms: hidden, inner and a gradient's tokens, and both sides of a
# matrix to orthogonalise that has more than 64 rows and columns.


def fsdp_operators_status(stream=None):
    """1 when a wait inside a kernel of the operators below has run out since
    the last question (their results are then undefined), else 0. Synchronises
    the stream."""
    v = ctypes.c_int(0)
    _check(lib().fsdp_operators_status(_stream(stream), ctypes.byref(v)))
    return v.value


def _whole(what, bits, **numbers):
    """Numbers that the C ABI's types would cut, and stand for others then, are refused."""
    for name, n in numbers.items():
        if not hasattr(n, "__index__"):
            _refuse(what, f"{name} {n!r} is no whole number")
        if not -(1 << bits - 1) <= n < 1 << bits - 1:
            _refuse(what, f"{name} {n} does not fit {bits} bits")


def _aligned(hidden, inner, aligned):
    return int(hidden % 8 == 0 and inner % 8 == 0) if aligned is None else int(bool(aligned))


def fsdp_gated_ffn_workspace(tokens, hidden, inner, aligned=None):
    """Bytes of the workspace that fsdp_gated_ffn needs for that many tokens or
    fewer. aligned: whether the rows of all its matrices start on the 16-byte
    grid, as contiguous ones do where hidden and inner are multiples of 8 (the
    default: whether they are)."""
    _whole("gated_ffn_workspace", 64, tokens=tokens, hidden=hidden, inner=inner)
    b = ctypes.c_size_t()
    _check(lib().fsdp_gated_ffn_workspace(tokens, hidden, inner, _aligned(hidden, inner, aligned), ctypes.byref(b)))
    return b.value


def _activation(what, name):
    act = ACTIVATIONS.get(name) if isinstance(name, str) else name
    if isinstance(act, bool) or not isinstance(act, int) or act not in ACTIVATIONS.values():
        _refuse(what, f"activation {name!r} is none of {sorted(ACTIVATIONS)}")
    return act


def fsdp_gated_ffn(x, w_gate, w_up, w_down, out, workspace, activation="silu", gate=None, up=None, stream=None):
    """out = (act(x w_gate^T) * (x w_up^T)) w_down^T. x, out: (tokens, hidden);
    w_gate, w_up: (inner, hidden); w_down: (hidden, inner); gate and up, both or
    neither given, receive the two projections (tokens, inner), which the
    gradient needs. activation: "silu", "gelu" or "relu". workspace: a tensor of
    at least fsdp_gated_ffn_workspace(tokens, hidden, inner) bytes."""
    what = "gated_ffn"
    act = _activation(what, activation)
    xp, rows, cols, xs, dt, dev = _matrix(what, "x", x)
    if dt != FSDP_BF16:
        _refuse(what, f"x is {x.dtype}; expected bfloat16")
    gp, inner, gcols, gs, _, _ = _matrix(what, "w_gate", w_gate)
    _like(what, "w_gate", w_gate, inner, cols, dt, dev)
    up_, us = _like(what, "w_up", w_up, inner, cols, dt, dev)
    dp, ds = _like(what, "w_down", w_down, cols, inner, dt, dev)
    kg, kgs = _like(what, "gate", gate, rows, inner, dt, dev)
    ku, kus = _like(what, "up", up, rows, inner, dt, dev)
    if (gate is None) != (up is None):
        _refuse(what, "gate and up: one of them is None")
    op, os_ = _like(what, "out", out, rows, cols, dt, dev)
    wp, wb = _work(what, workspace, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_gated_ffn(rows, cols, inner, xp, xs, gp, gs, up_, us, dp, ds, act, kg, kgs, ku, kus, op, os_, wp, wb,
                                handle))


def fsdp_gated_ffn_grad_workspace(tokens, hidden, inner, aligned=None):
    """Bytes of the workspace that fsdp_gated_ffn_grad needs, as fsdp_gated_ffn_workspace."""
    _whole("gated_ffn_grad_workspace", 64, tokens=tokens, hidden=hidden, inner=inner)
    b = ctypes.c_size_t()
    _check(lib().fsdp_gated_ffn_grad_workspace(tokens, hidden, inner, _aligned(hidden, inner, aligned), ctypes.byref(b)))
    return b.value


def fsdp_gated_ffn_grad(grad_out, x, w_gate, w_up, w_down, gate, up, grad_x, grad_w_gate, grad_w_up, grad_w_down, workspace,
                        activation="silu", accumulate=False, stream=None):
    """Gradient of fsdp_gated_ffn from the gate and up that it gave: grad_x and
    the three weights' gradients, float32 or bfloat16 (with accumulate, added to
    what they hold). workspace: a tensor of at least
    fsdp_gated_ffn_grad_workspace(tokens, hidden, inner) bytes."""
    what = "gated_ffn_grad"
    act = _activation(what, activation)
    gp, rows, cols, gs, dt, dev = _matrix(what, "grad_out", grad_out)
    if dt != FSDP_BF16:
        _refuse(what, f"grad_out is {grad_out.dtype}; expected bfloat16")
    xp, xs = _like(what, "x", x, rows, cols, dt, dev)
    wgp, inner, _, wgs, _, _ = _matrix(what, "w_gate", w_gate)
    _like(what, "w_gate", w_gate, inner, cols, dt, dev)
    wup, wus = _like(what, "w_up", w_up, inner, cols, dt, dev)
    wdp, wds = _like(what, "w_down", w_down, cols, inner, dt, dev)
    kg, kgs = _like(what, "gate", gate, rows, inner, dt, dev)
    ku, kus = _like(what, "up", up, rows, inner, dt, dev)
    dxp, dxs = _like(what, "grad_x", grad_x, rows, cols, dt, dev)
    pdt = (_TYPES or _types()).get(grad_w_gate.dtype)
    dgp, dgs = _like(what, "grad_w_gate", grad_w_gate, inner, cols, pdt, dev)
    dup, dus = _like(what, "grad_w_up", grad_w_up, inner, cols, pdt, dev)
    ddp, dds = _like(what, "grad_w_down", grad_w_down, cols, inner, pdt, dev)
    wp, wb = _work(what, workspace, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_gated_ffn_grad(rows, cols, inner, gp, gs, xp, xs, wgp, wgs, wup, wus, wdp, wds, kg, kgs, ku, kus, act, dxp,
                                     dxs, pdt, int(accumulate), dgp, dgs, dup, dus, ddp, dds, wp, wb, handle))


def fsdp_orthogonalize_workspace(rows, cols):
    """Bytes of the workspace that fsdp_orthogonalize needs."""
    _whole("orthogonalize_workspace", 64, rows=rows, cols=cols)
    b = ctypes.c_size_t()
    _check(lib().fsdp_orthogonalize_workspace(rows, cols, ctypes.byref(b)))
    return b.value


def fsdp_orthogonalize(x, out, workspace, steps=5, coefficients=(3.4445, -4.7750, 2.0315), scale=1.0, eps=1e-7, stream=None):
    """out = scale * X after `steps` Newton-Schulz steps from X = x / (|x| + eps):
    with A = X X^T, X <- a X + (b A + c A A) X. x: a matrix of float32 or
    bfloat16; out: the same shape in bfloat16. The coefficients have to keep
    singular values that start in [0, 1] at or below 8 until the last step.
    workspace: a tensor of at least fsdp_orthogonalize_workspace(rows, cols)
    bytes."""
    what = "orthogonalize"
    _whole(what, 32, steps=steps)
    xp, rows, cols, xs, dt, dev = _matrix(what, "x", x)
    op, os_ = _like(what, "out", out, rows, cols, FSDP_BF16, dev)
    a, b, c = coefficients
    wp, wb = _work(what, workspace, dev)
    handle = _on(what, dev, stream)
    _check(lib().fsdp_orthogonalize(rows, cols, dt, xp, xs, steps, a, b, c, scale, eps, op, os_, wp, wb, handle))
