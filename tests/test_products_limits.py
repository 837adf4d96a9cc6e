"""The longest sums that the products' calls take, without a GPU."""
import ctypes

import pytest

from hsdp_sharded_parameter_gb300 import capi as C
from test_products_host import P, ffn, grad, ortho, refused

LONG = 2 ** 24


@pytest.mark.parametrize("change", [dict(h=LONG + 1, xs=LONG + 8, wgs=LONG + 8, wus=LONG + 8, os=LONG + 8), dict(f=LONG + 1, wds=LONG + 8)])
def test_gated_ffn(change):
    refused(ffn(**change), "sum", "2^24")
    # as many tokens as ever: a token is no term of a sum
    refused(ffn(t=LONG + 1, wb=0), "workspace", "needs")


@pytest.mark.parametrize("change", [dict(t=LONG + 1), dict(h=LONG + 1, dys=LONG + 8, xs=LONG + 8, wgs=LONG + 8, wus=LONG + 8, dxs=LONG + 8, dgs=LONG + 8,
                                                          dus=LONG + 8), dict(f=LONG + 1, wds=LONG + 8, gs=LONG + 8, us=LONG + 8, dds=LONG + 8)])
def test_gated_ffn_grad(change):
    refused(grad(**change), "sum", "2^24")
    refused(grad(t=LONG, wb=0), "workspace", "needs")


def test_orthogonalize():
    refused(ortho(r=65, c=LONG + 1, xs=LONG + 1, os=LONG + 1), "sum", "2^24")
    refused(ortho(r=LONG + 1, c=65, xs=65, os=65), "sum", "2^24")
    for r, c in [(64, LONG + 1), (LONG + 1, 64), (65, LONG), (LONG, 65)]:
        refused(ortho(r=r, c=c, xs=c, os=c, wb=0), "workspace", "needs")


def test_workspaces():
    b = ctypes.byref(ctypes.c_size_t())
    L = C.lib()
    for args in [(8, LONG + 1, 8), (8, 8, LONG + 1)]:
        refused(L.fsdp_gated_ffn_workspace(*args, 1, b), "sum", "2^24")
    for args in [(LONG + 1, 8, 8), (8, LONG + 1, 8), (8, 8, LONG + 1)]:
        refused(L.fsdp_gated_ffn_grad_workspace(*args, 1, b), "sum", "2^24")
    refused(L.fsdp_orthogonalize_workspace(65, LONG + 1, b), "sum", "2^24")
    assert L.fsdp_gated_ffn_workspace(LONG + 1, 8, 8, 1, b) == C.FSDP_OK
    assert L.fsdp_orthogonalize_workspace(64, 2 ** 31 - 513, b) == C.FSDP_OK


def test_operands_without_elements_overlap_nothing():
    # no tokens, or no columns, on views of one buffer
    assert ffn(t=0, x=P, out=P, g=P, gs=16, u=P, us=16, work=None, wb=0) == C.FSDP_OK
    assert ffn(t=0, h=0, x=P, wg=P, wu=P, wd=P, out=P, work=None, wb=0) == C.FSDP_OK
    assert ortho(r=0, x=P, out=P, work=None, wb=0) == C.FSDP_OK
    assert ortho(c=0, x=P, out=P, work=None, wb=0) == C.FSDP_OK
    # those that hold elements do
    refused(ffn(t=1, x=P, out=P), "out", "another operand")
    refused(ffn(t=3, f=0, g=P, u=P, out=P), "out", "another operand")
    refused(grad(t=0, dg=9 * P, du=9 * P), "another operand")
