"""The training operators' host side, without a GPU: the generator against its
published answers, the mask's shape, and the refusals of the C ABI and of the
binding, all of which come before anything is enqueued."""
import ctypes
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import operators_ref as R
from hsdp_sharded_parameter_gb300 import capi as C

P = 1 << 20  # a pointer that no refused call follows


def test_philox_known_answers():
    # the known-answer vectors published with the generator (philox4x32, 10 rounds)
    for ctr, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(x) for x in R.philox(*ctr, *key)) == want


def test_mask_is_a_function_of_row_and_column():
    m = R.mask(40, 100, 0.25, 0x123456789ABCDEF, 7)
    assert np.array_equal(m[5:9, :33], R.mask(4, 33, 0.25, 0x123456789ABCDEF, 7, first_row=5))
    k = R.limit(0.25)
    assert set(np.unique(m)) == {0.0, 65536.0 / k}
    assert abs((m > 0).mean() - 0.75) < 6 * math.sqrt(0.75 * 0.25 / m.size)
    assert not np.array_equal(m, R.mask(40, 100, 0.25, 0x123456789ABCDEF, 8))


def refused(rc, *words):
    assert rc == C.FSDP_ERR_INVALID_ARG
    msg = C.lib().fsdp_last_error().decode()
    assert all(w in msg for w in words), msg


def emb(**k):
    a = dict(tdt=0, table=P, ts=8, vocab=4, cols=8, it=1, ids=P, n=3, first=0, scale=1.0, odt=0, out=2 * P, os=8)
    a.update(k)
    return C.lib().fsdp_embedding(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(tdt=2), ["table", "dtype"]), (dict(table=None), ["table", "NULL"]), (dict(table=P + 2), ["table", "aligned"]),
    (dict(ts=-1), ["table", "stride"]), (dict(vocab=-1), ["vocab"]), (dict(vocab=2 ** 31), ["vocab"]), (dict(cols=-1), ["size"]),
    (dict(it=2), ["index type"]), (dict(ids=None), ["ids"]), (dict(ids=P + 4), ["ids", "aligned"]), (dict(n=-1), ["n_ids"]),
    (dict(n=2 ** 31), ["n_ids"]), (dict(scale=math.nan), ["scale"]), (dict(scale=1e300), ["scale"]), (dict(odt=-1), ["out"]),
    (dict(out=None), ["out", "NULL"]), (dict(os=7), ["out", "overlap"]), (dict(ts=2 ** 62), ["table", "stride"])])
def test_embedding_refuses(change, words):
    refused(emb(**change), *words)


def emb_grad(**k):
    a = dict(gdt=0, grad=P, gs=8, it=0, ids=P, n=3, first=0, scale=1.0, acc=0, tdt=1, table=2 * P, ts=8, vocab=4, cols=8,
             work=3 * P, wb=C.fsdp_embedding_grad_workspace(3, 4, 8))
    a.update(k)
    return C.lib().fsdp_embedding_grad(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(gdt=3), ["grad_out"]), (dict(grad=None), ["grad_out", "NULL"]), (dict(table=2 * P + 1), ["grad_table", "aligned"]),
    (dict(ts=4), ["grad_table", "overlap"]), (dict(table=None), ["grad_table"]), (dict(work=None), ["workspace"]),
    (dict(work=3 * P + 8), ["workspace", "aligned"]), (dict(wb=8), ["workspace", "needs"]), (dict(scale=math.inf), ["scale"]),
    (dict(ids=P + 2), ["ids"])])
def test_embedding_grad_refuses(change, words):
    refused(emb_grad(**change), *words)


def drop(**k):
    a = dict(rows=3, cols=8, dt=1, x=P, xs=8, res=None, rs=0, p=0.5, seed=1, draw=0, out=2 * P, os=8)
    a.update(k)
    return C.lib().fsdp_dropout(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(rows=-1), ["size"]), (dict(cols=2 ** 34 + 1, rows=1, os=2 ** 35), ["columns"]), (dict(dt=9), ["dtype"]),
    (dict(x=None), ["x", "NULL"]), (dict(x=P + 1), ["aligned"]), (dict(p=-0.1), ["p "]), (dict(p=1.5), ["p "]),
    (dict(p=math.nan), ["p "]), (dict(os=4), ["overlap"]), (dict(out=P, os=16), ["another stride"]),
    (dict(res=2 * P, rs=9), ["another stride"]), (dict(rows=2 ** 30, xs=2 ** 40), ["too large"])])
def test_dropout_refuses(change, words):
    refused(drop(**change), *words)


def norm(**k):
    a = dict(rows=3, cols=8, dt=1, x=P, xs=8, res=None, rs=0, p=0.0, seed=1, draw=0, pdt=0, w=2 * P, b=None, eps=1e-5,
             hidden=None, hs=0, out=3 * P, os=8, mean=4 * P, rstd=None)
    a.update(k)
    return C.lib().fsdp_layer_norm(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(rows=2 ** 31), ["rows"]), (dict(out=P), ["out"]), (dict(hidden=P, hs=8), ["hidden"]),
    (dict(hidden=3 * P, hs=8), ["out"]), (dict(mean=4 * P + 2), ["mean"]), (dict(rstd=1), ["rstd"]), (dict(eps=-1.0), ["eps"]),
    (dict(eps=math.nan), ["eps"]), (dict(w=2 * P + 1), ["weight"]), (dict(pdt=5), ["weight", "dtype"]), (dict(out=None), ["out"]),
    (dict(hidden=5 * P, hs=7), ["hidden", "overlap"]), (dict(p=2.0), ["p "])])
def test_layer_norm_refuses(change, words):
    refused(norm(**change), *words)


def norm_grad(**k):
    a = dict(rows=3, cols=8, dt=1, grad=P, gs=8, gh=None, ghs=0, hidden=2 * P, hs=8, mean=3 * P, rstd=3 * P, pdt=0, w=None,
             p=0.0, seed=1, draw=0, acc=0, res=None, rs=0, x=4 * P, xs=8, gdt=0, gw=5 * P, gb=None, work=6 * P,
             wb=C.fsdp_layer_norm_grad_workspace(3, 8))
    a.update(k)
    return C.lib().fsdp_layer_norm_grad(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(grad=None), ["grad_out"]), (dict(hidden=None), ["hidden"]), (dict(mean=None), ["mean"]), (dict(rstd=None), ["rstd"]),
    (dict(x=P), ["grad_x"]), (dict(x=2 * P), ["grad_x"]), (dict(res=4 * P, rs=8), ["grad_x"]), (dict(res=P, rs=8), ["grad_residual"]),
    (dict(wb=0), ["workspace"]), (dict(work=6 * P + 4), ["workspace"]), (dict(gdt=7), ["grad_weight"]), (dict(gb=2), ["grad_bias"]),
    (dict(xs=3), ["grad_x", "overlap"]), (dict(p=-1.0), ["p "]), (dict(rows=-2), ["size"])])
def test_layer_norm_grad_refuses(change, words):
    refused(norm_grad(**change), *words)


def test_workspace_queries():
    b = ctypes.c_size_t()
    refused(C.lib().fsdp_embedding_grad_workspace(-1, 4, 8, ctypes.byref(b)))
    refused(C.lib().fsdp_embedding_grad_workspace(1, 4, 8, None), "NULL")
    refused(C.lib().fsdp_embedding_grad_workspace(1, 4, 2 ** 31, ctypes.byref(b)), "columns")
    refused(C.lib().fsdp_layer_norm_grad_workspace(1, -8, ctypes.byref(b)))
    assert C.fsdp_layer_norm_grad_workspace(0, 100) == 0
    # no more than a few times what the operators read
    assert C.fsdp_embedding_grad_workspace(65536, 131072, 8192) < 65536 * 8192 * 4
    assert C.fsdp_layer_norm_grad_workspace(16384, 8192) < 16384 * 8192


def test_nothing_to_do_needs_no_gpu():
    before = C.fsdp_launch_count()
    assert emb(n=0, ids=None, table=None, out=None) == C.FSDP_OK
    assert emb(cols=0) == C.FSDP_OK
    assert drop(rows=0) == C.FSDP_OK and drop(cols=0, x=None, out=None) == C.FSDP_OK
    assert norm(rows=0, x=None, out=None) == C.FSDP_OK
    assert emb_grad(vocab=0, table=None, wb=1 << 20) == C.FSDP_OK
    assert emb_grad(n=0, acc=1, wb=1 << 20) == C.FSDP_OK
    assert norm_grad(cols=0) == C.FSDP_OK
    assert C.fsdp_launch_count() == before


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in [lambda: C.fsdp_dropout(x, x, 0.5, 1), lambda: C.fsdp_embedding(x, ids, x),
                 lambda: C.fsdp_embedding_grad(x, ids, x, x), lambda: C.fsdp_layer_norm(x, None, None, x, None, None),
                 lambda: C.fsdp_layer_norm_grad(x, x, x, x, None, x, None, None, x)]:
        with pytest.raises(C.FsdpError) as e:
            call()
        assert e.value.code == C.FSDP_ERR_INVALID_ARG


@pytest.mark.parametrize("cols", [16384, 16385, 16640, 40000, 2 ** 34, 2 ** 40])
def test_layer_norm_grad_workspace_of_wide_rows(cols):
    # in a process of its own: an integer division by zero ends the process on some hosts
    code = f"from hsdp_sharded_parameter_gb300 import capi as C; print(C.fsdp_layer_norm_grad_workspace(4, {cols}))"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert int(r.stdout) == 4 * 2 * (-(-cols // 8) * 8) * 4  # a part a row, weight and bias
    # the call asks the same question first
    if cols <= 2 ** 34:
        refused(norm_grad(cols=cols, gs=cols, hs=cols, xs=cols, wb=0), "workspace", "needs")


@pytest.mark.parametrize("cols", [8, 256, 5000, 40000])
def test_a_workspace_serves_smaller_calls(cols):
    # across every number of tokens at which the gradient's chunks grow, whatever the GPU
    sizes = list(range(0, 600)) + list(range(600, 21000, 61)) + [4096, 4097, 16384, 16385, 65536, 10 ** 6]
    got = [C.fsdp_embedding_grad_workspace(n, 32000, cols) for n in sorted(sizes)]
    assert got == sorted(got)
    for n in (1, 700, 20000):
        got = [C.fsdp_embedding_grad_workspace(n, v, cols) for v in (0, 1, 31, 33, 4099, 32000, 131072)]
        assert got == sorted(got)
    got = [C.fsdp_layer_norm_grad_workspace(r, cols) for r in range(0, 6000)]
    assert got == sorted(got)


@pytest.mark.parametrize("n", [2 ** 31 - 2 ** 14, 2 ** 31 - 8192, 2 ** 31 - 2])
def test_embedding_grad_refuses_tokens_that_its_sort_cannot_number(n):
    # a step of 8192 tokens past the last one, and the next, have to fit 32 bits with a sign
    refused(emb_grad(n=n, wb=2 ** 62), "n_ids")
    b = ctypes.c_size_t()
    refused(C.lib().fsdp_embedding_grad_workspace(n, 4, 8, ctypes.byref(b)), "n_ids")


def test_embedding_grad_takes_as_many_tokens_as_the_header_says():
    n = 2 ** 31 - 2 ** 14 - 1
    assert C.fsdp_embedding_grad_workspace(n, 4, 8) > 16 * n  # two buffers of (row, token)
    refused(emb_grad(n=n, wb=16 * n), "workspace", "needs")


class OnGpu:
    """What the binding asks of a 4 x 8 float32 tensor on the first GPU."""
    dtype, is_cuda, shape, device = torch.float32, True, (4, 8), "cuda:0"
    stride, data_ptr, get_device = (lambda self: (8, 1)), (lambda self: P), (lambda self: 0)


def test_first_calls_from_several_threads(monkeypatch):
    # a second thread's first call, made between any two lines of the first
    # thread's as soon as there is something in the table
    monkeypatch.setattr(C, "_TYPES", {})
    want, seen = (P, 4, 8, 8, C.FSDP_F32, 0), []

    def second():
        sys.settrace(None)  # of this thread
        try:
            seen.append(C._matrix("test", "x", OnGpu()))
        except Exception as e:
            seen.append(e)

    def trace(frame, event, arg):
        if frame.f_code is not C._types.__code__:
            return None
        if not C._TYPES:
            return trace
        t = threading.Thread(target=second)
        t.start()
        t.join(30)
        return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        got = C._matrix("test", "x", OnGpu())
    finally:
        sys.settrace(old)
    assert got == want and seen and all(s == want for s in seen), seen


@pytest.mark.parametrize("change, word", [(dict(draw=2 ** 32), "draw"), (dict(draw=-(2 ** 31) - 1), "draw"), (dict(seed=2 ** 64), "seed"),
                                          (dict(seed=-(2 ** 63) - 1), "seed")])
def test_binding_refuses_numbers_that_a_mask_would_cut(change, word):
    # 2^32 would draw the mask of 0 again
    x, a = torch.zeros(4, 8), dict(p=0.5, seed=1, draw=0)
    a.update(change)
    for call in [lambda: C.fsdp_dropout(x, x, **a), lambda: C.fsdp_layer_norm(x, None, None, x, None, None, **a),
                 lambda: C.fsdp_layer_norm_grad(x, x, x, x, None, x, None, None, x, **a)]:
        with pytest.raises(C.FsdpError, match=word) as e:
            call()
        assert e.value.code == C.FSDP_ERR_INVALID_ARG


def test_binding_refuses_a_first_row_that_would_be_cut():
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for first in (2 ** 63, 2 ** 64 + 5, -(2 ** 63) - 1):
        for call in [lambda: C.fsdp_embedding(x, ids, x, first_row=first), lambda: C.fsdp_embedding_grad(x, ids, x, x, first_row=first)]:
            with pytest.raises(C.FsdpError, match="first_row"):
                call()
