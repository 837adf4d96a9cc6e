"""Numbers that the C ABI's types would cut are refused by the binding, without a GPU."""
import pytest
import torch

from hsdp_sharded_parameter_gb300 import capi as C


@pytest.mark.parametrize("steps", [2 ** 32 + 5, -2 ** 32 + 5, 2 ** 64 + 1, 5.0, "5", None])
def test_steps(steps):
    x = torch.zeros(4, 8)
    with pytest.raises(C.FsdpError, match="steps"):
        C.fsdp_orthogonalize(x, x, x, steps=steps)


@pytest.mark.parametrize("activation", [2 ** 32, 3, -1, "swish", None, 1.0, [], True])
def test_activation(activation):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(C.FsdpError, match="activation"):
        C.fsdp_gated_ffn(x, x, x, x, x, x, activation)
    with pytest.raises(C.FsdpError, match="activation"):
        C.fsdp_gated_ffn_grad(x, x, x, x, x, x, x, x, x, x, x, x, activation)


def test_activations_by_number():
    # the C ABI's own numbers are taken as they were: the refusal is of the tensors
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for activation in (C.FSDP_SILU, C.FSDP_GELU, C.FSDP_RELU, "silu", "gelu", "relu"):
        with pytest.raises(C.FsdpError, match="GPU"):
            C.fsdp_gated_ffn(x, x, x, x, x, x, activation)


@pytest.mark.parametrize("n", [2 ** 64 + 5, 2 ** 63, -2 ** 64 + 5, 5.0])
def test_workspaces(n):
    for call in (lambda: C.fsdp_gated_ffn_workspace(n, 8, 8), lambda: C.fsdp_gated_ffn_workspace(8, n, 8), lambda: C.fsdp_gated_ffn_workspace(8, 8, n),
                 lambda: C.fsdp_gated_ffn_grad_workspace(n, 8, 8), lambda: C.fsdp_gated_ffn_grad_workspace(8, n, 8),
                 lambda: C.fsdp_gated_ffn_grad_workspace(8, 8, n, aligned=True), lambda: C.fsdp_orthogonalize_workspace(n, 8),
                 lambda: C.fsdp_orthogonalize_workspace(8, n)):
        with pytest.raises(C.FsdpError, match="64 bits|whole"):
            call()
