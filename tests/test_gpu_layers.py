"""TokenBlock: the training operators together on an HSDP mesh, against the
same block in 64 bits with autograd, and the example's loss."""
import os
import sys

import numpy as np
import pytest
import torch

import operators_ref as R
from hsdp_sharded_parameter_gb300.layers import TokenBlock

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(block, ids, grad_out, step):
    """(out, gradients averaged over the ranks) in 64 bits, on the CPU."""
    outs, total = [], None
    for w in range(block.plan.W):
        par = [torch.from_numpy(R.f64(t)).requires_grad_() for t in block._views(block.unit.full, w)]
        d0, d1 = block._draws(step, w)
        k0, k1 = (torch.from_numpy(R.mask(block.tokens, block.hidden, block.p, block.seed, d)) for d in (d0, d1))
        i = ids[w].cpu()
        named = (i >= 0) & (i < block.vocab)
        e = torch.where(named[:, None], block.scale * par[0][i.clamp(0, block.vocab - 1)], 0.0)
        h = k0 * e
        n = torch.nn.functional.layer_norm(h, (block.hidden,), par[1], par[2], block.eps)
        out = h + k1 * (n @ par[3].t())
        outs.append(out.detach())
        g = torch.autograd.grad((out * torch.from_numpy(R.f64(grad_out[w]))).sum(), par)
        total = list(g) if total is None else [a + b for a, b in zip(total, g)]
    return outs, [t / block.plan.W for t in total]


@pytest.mark.parametrize("dtype, tol", [("f32", 1e-4), ("bf16", 0.05)])
def test_token_block_against_64_bits(dtype, tol):
    # tol, relative to each output's root mean square: about 20 binary32 (or a
    # few bfloat16, each 2^-8) roundings in a chain through a product of 48
    # terms; the mesh's reduction adds one more rounding. torch may take TF32
    # for nothing here: products of fp32 are asked for in full.
    torch.backends.cuda.matmul.allow_tf32 = False
    block = TokenBlock(50, 48, 70, 4, 2, dtype=dtype, p=0.25, seed=99)
    block.init_parameters(3, std=0.3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    ids = [torch.randint(-2, 52, (70,), generator=gen, device="cuda") for _ in range(4)]
    grad = [torch.randn(70, 48, generator=gen, device="cuda").to(block.out[0].dtype) for _ in range(4)]
    for step in (0, 7):
        out = block.forward(ids, step)
        block.backward(ids, grad, step)
        want, grads = reference(block, ids, grad, step)
        for w in range(4):
            assert np.abs(R.f64(out[w]) - want[w].numpy()).max() <= tol * max(1.0, float(want[w].abs().max()))
        for w in range(4):
            for q in range(4):
                first, n = block.plan.sharded_size(q, w % 2)
                ref = grads[q][first:first + n].reshape(-1).numpy()
                got = R.f64(block.unit.shard_grads[w * 4 + q])
                rms = np.sqrt(np.mean(ref ** 2)) if ref.size else 0.0
                assert np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref) + 1e-12, (q, w)
                assert np.abs(got - ref).max(initial=0.0) <= 20 * tol * rms
    block.close()


def test_steps_draw_masks_of_their_own_and_repeat():
    block = TokenBlock(40, 64, 33, 2, 2, dtype="bf16", p=0.5, seed=4)
    block.init_parameters(1)
    ids = [torch.arange(33, device="cuda") for _ in range(2)]
    a = [t.clone() for t in block.forward(ids, 3)]
    assert not torch.equal(a[0], a[1])  # ranks
    b = [t.clone() for t in block.forward(ids, 4)]
    assert not torch.equal(a[0], b[0])  # steps
    assert all(torch.equal(x, y) for x, y in zip(block.forward(ids, 3), a))
    block.close()


def test_example_trains():
    from train_token_block import train

    losses = train(steps=30, vocab=500, hidden=128, tokens=256, rank_size=4, shard_size=2, say=None)
    assert all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0], losses
