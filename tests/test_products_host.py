"""The products' operators' host side, without a GPU: the refusals of the C ABI
and of the binding, which come before anything is enqueued, and the workspaces'
sizes."""
import ctypes
import math

import pytest
import torch

import products_ref as R
from hsdp_sharded_parameter_gb300 import capi as C

P = 1 << 20  # a pointer that no refused call follows


def refused(rc, *words):
    assert rc == C.FSDP_ERR_INVALID_ARG
    msg = C.lib().fsdp_last_error().decode()
    assert all(w in msg for w in words), msg


def ffn(**k):
    a = dict(t=3, h=8, f=16, x=P, xs=8, wg=2 * P, wgs=8, wu=3 * P, wus=8, wd=4 * P, wds=16, act=0, g=None, gs=0, u=None, us=0,
             out=5 * P, os=8, work=6 * P, wb=1 << 24)
    a.update(k)
    return C.lib().fsdp_gated_ffn(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(t=-1), ["size"]), (dict(h=2 ** 31), ["size"]), (dict(f=2 ** 31 - 1), ["size"]), (dict(act=3), ["activation"]),
    (dict(x=None), ["x", "NULL"]), (dict(x=P + 1), ["x", "aligned"]), (dict(wgs=-8), ["w_gate", "stride"]), (dict(wu=None), ["w_up"]),
    (dict(wd=None), ["w_down"]), (dict(g=7 * P, gs=16), ["gate and up"]), (dict(u=7 * P, us=16), ["gate and up"]),
    (dict(g=7 * P, gs=15, u=8 * P, us=16), ["gate", "overlap"]), (dict(g=7 * P, gs=16, u=7 * P, us=16), ["another operand"]),
    (dict(out=P), ["out", "another operand"]), (dict(os=7), ["out", "overlap"]), (dict(out=None), ["out"]), (dict(wb=8), ["workspace", "needs"]),
    (dict(work=None), ["workspace"]), (dict(work=6 * P + 8), ["workspace", "aligned"])])
def test_gated_ffn_refuses(change, words):
    refused(ffn(**change), *words)


def grad(**k):
    a = dict(t=3, h=8, f=16, dy=P, dys=8, x=2 * P, xs=8, wg=3 * P, wgs=8, wu=4 * P, wus=8, wd=5 * P, wds=16, g=6 * P, gs=16, u=7 * P, us=16,
             act=1, dx=8 * P, dxs=8, dt=0, acc=0, dg=9 * P, dgs=8, du=10 * P, dus=8, dd=11 * P, dds=16, work=12 * P, wb=1 << 24)
    a.update(k)
    return C.lib().fsdp_gated_ffn_grad(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(t=-1), ["size"]), (dict(act=-1), ["activation"]), (dict(g=None), ["gate"]), (dict(u=None), ["up"]), (dict(dt=2), ["dtype"]),
    (dict(dx=P), ["grad_x", "another operand"]), (dict(du=9 * P), ["another operand"]), (dict(dd=5 * P), ["grad_w_down", "another operand"]),
    (dict(dds=15), ["grad_w_down", "overlap"]), (dict(dg=9 * P + 2), ["grad_w_gate", "aligned"]), (dict(wb=100), ["workspace", "needs"]),
    (dict(dx=None), ["grad_x"]), (dict(dd=None), ["grad_w_down"])])
def test_gated_ffn_grad_refuses(change, words):
    refused(grad(**change), *words)


def ortho(**k):
    a = dict(r=70, c=90, dt=0, x=P, xs=90, steps=5, a=3.4445, b=-4.775, k=2.0315, scale=1.0, eps=1e-7, out=2 * P, os=90, work=3 * P, wb=1 << 24)
    a.update(k)
    return C.lib().fsdp_orthogonalize(*a.values(), None)


@pytest.mark.parametrize("change, words", [
    (dict(r=-1), ["size"]), (dict(dt=2), ["dtype"]), (dict(x=None), ["x"]), (dict(steps=0), ["steps"]), (dict(steps=65), ["steps"]),
    (dict(a=math.nan), ["coefficient"]), (dict(b=-257.0), ["coefficient"]), (dict(k=math.inf), ["coefficient"]), (dict(scale=math.inf), ["scale"]),
    (dict(eps=-1.0), ["eps"]), (dict(eps=math.nan), ["eps"]), (dict(out=P), ["out", "another operand"]), (dict(os=89), ["out", "overlap"]),
    (dict(wb=64), ["workspace", "needs"])])
def test_orthogonalize_refuses(change, words):
    refused(ortho(**change), *words)


def test_workspaces():
    b = ctypes.c_size_t()
    refused(C.lib().fsdp_gated_ffn_workspace(1, 8, 8, 1, None), "NULL")
    refused(C.lib().fsdp_gated_ffn_grad_workspace(-1, 8, 8, 1, ctypes.byref(b)), "size")
    refused(C.lib().fsdp_orthogonalize_workspace(2 ** 31, 8, ctypes.byref(b)), "size")
    refused(C.lib().fsdp_operators_status(None, None), "NULL")
    for f in (C.fsdp_gated_ffn_workspace, C.fsdp_gated_ffn_grad_workspace):
        for hidden, inner in [(4096, 11008), (17, 5), (136, 4000)]:
            for aligned in (True, False):
                got = [f(t, hidden, inner, aligned) for t in list(range(0, 700)) + list(range(700, 20000, 97))]
                assert got == sorted(got)
            assert f(64, hidden, inner) in (f(64, hidden, inner, True), f(64, hidden, inner, False))
    # a call of fewer tokens finds enough in a larger one's workspace: the refusal says what it needs
    for t in range(1, 600, 7):
        for h, f in [(64, 128), (512, 1376), (4096, 64)]:
            need = C.fsdp_gated_ffn_workspace(600, h, f)
            ffn(t=t, h=h, f=f, xs=h, wgs=h, wus=h, wds=f, os=h, wb=0)
            msg = C.lib().fsdp_last_error().decode()
            assert int(msg.split("needs ")[1]) <= min(need, C.fsdp_gated_ffn_workspace(t, h, f))


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in [lambda: C.fsdp_gated_ffn(x, x, x, x, x, x), lambda: C.fsdp_gated_ffn_grad(x, x, x, x, x, x, x, x, x, x, x, x),
                 lambda: C.fsdp_orthogonalize(x, x, x)]:
        with pytest.raises(C.FsdpError) as e:
            call()
        assert e.value.code == C.FSDP_ERR_INVALID_ARG


def test_the_references_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wg, wu, wd, dy = r(5, 6), r(7, 6), r(7, 6), r(6, 7), r(5, 6)
    for act in ("silu", "gelu", "relu"):
        y = lambda x, wg, wu, wd: float((((R.act(act, x @ wg.T)[0] * (x @ wu.T)) @ wd.T) * dy).sum())  # noqa: E731
        want = R.gated_ffn_grad(dy, x, wg, wu, wd, x @ wg.T, x @ wu.T, act)
        for i, name in enumerate(("x", "w_gate", "w_up", "w_down")):
            args = [x, wg, wu, wd]
            step = r(*args[i].shape) * 1e-6
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + step, args[i] - step
            # off by the third derivative times step^2 and by 2^-52 of the sums over the step
            assert abs((y(*up) - y(*down)) / 2 - float((want[name][0] * step).sum())) < 1e-9
