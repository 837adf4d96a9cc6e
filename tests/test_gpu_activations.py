"""The activations of the gated block and their slopes value by value, far into
their tails, against 64 bits.

With one token each, or with unit factors, the block's outputs are the
activation's values rounded to bfloat16 on the way (h, the gradient of gate) and
once more at the end: 2 * 2^-8 of the value. Before that they are off by a few
roundings of binary32. An argument of exp or erfc that is rounded moves their
values by 2^-24 of it times their relative slope, at most z^2 at z: (z^2 + 16) *
2^-23 of the value covers it and the functions' own errors. A slope is a sum of
two terms that cancel where it is 0: what is relative to a value above is
relative to the terms there. Below the smallest normal number, 2^-126, values
may go their own ways."""
import pytest
import torch

from hsdp_sharded_parameter_gb300 import capi as C

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
Z = torch.cat([torch.linspace(-110, 110, 881), torch.linspace(-16, 16, 2049), torch.logspace(-36, 2, 200), -torch.logspace(-36, 2, 200),
               torch.zeros(1)]).to(BF16)


def formula(name, z):
    """Value, slope, and the size of the slope's terms."""
    z = z.double()
    if name == "silu":
        p = torch.where(z >= 0, 1 / (1 + torch.exp(-z)), torch.exp(z) / (1 + torch.exp(z)))
        q = torch.where(z >= 0, torch.exp(-z) / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z)))
        return z * p, p + z * p * q, p + (z * p * q).abs()
    if name == "gelu":
        p, d = 0.5 * torch.special.erfc(-z / 2 ** 0.5), z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
        return z * p, p + d, p + d.abs()
    return torch.clamp(z, min=0), (z > 0).double(), (z > 0).double()


def close(got, want, terms):
    z = Z.double()
    err = (2 * 2.0 ** -8 * 1.01 * want.abs() + (z * z + 16) * 2.0 ** -23 * terms + 2.0 ** -125 * (1 + z.abs()))
    bad = ~((got.double().cpu() - want).abs() <= err)
    assert not bool(bad.any()), [(float(a), float(b), float(c)) for a, b, c in zip(Z[bad][:8], got.cpu()[bad][:8], want[bad][:8])]


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_values(name):
    n = len(Z)
    x = torch.zeros(n, 8, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = Z.cuda(), 1
    w_gate, w_up = torch.zeros(8, 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda")
    w_gate[:, 0], w_up[:, 1] = 1, 1
    out, gate, up = (torch.empty_like(x) for _ in range(3))
    work = torch.empty(C.fsdp_gated_ffn_workspace(n, 8, 8), dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn(x, w_gate, w_up, torch.eye(8, dtype=BF16, device="cuda"), out, work, name, gate, up)
    assert torch.equal(gate, x[:, :1].expand(-1, 8)) and bool((up == 1).all())
    value, _, _ = formula(name, Z)
    assert torch.equal(out, out[:, :1].expand(-1, 8))
    close(out[:, 0], value, value.abs())


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_values_and_slopes_in_the_gradient(name):
    # one token, inner as long as Z: d = 1, so the gradient of gate is the slope and that of w_down the value
    n = len(Z)
    one = torch.zeros(1, 8, dtype=BF16, device="cuda")
    one[0, 0] = 1
    gate, up = Z.cuda()[None].contiguous(), torch.ones(1, n, dtype=BF16, device="cuda")
    w_down = torch.zeros(8, n, dtype=BF16, device="cuda")
    w_down[0] = 1
    w = torch.zeros(n, 8, dtype=BF16, device="cuda")
    grads = [torch.empty(n, 8, device="cuda"), torch.empty(n, 8, device="cuda"), torch.empty(8, n, device="cuda")]
    work = torch.empty(C.fsdp_gated_ffn_grad_workspace(1, 8, n, aligned=False), dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn_grad(one, one, w, w, w_down, gate, up, torch.empty_like(one), *grads, work, name)
    value, slope, terms = formula(name, Z)
    close(grads[0][:, 0], slope, terms)
    close(grads[1][:, 0], value, value.abs())
    close(grads[2][0], value, value.abs())
