"""Trains a TokenBlock on synthetic tokens: embedding, dropout, layer norm and
their gradients on an HSDP mesh, all virtual ranks on one GPU.

    python examples/train_token_block.py [--steps 50] [--vocab 32000] [--hidden 1024]

Each token has a fixed random target; the loss is the mean squared distance to
it over the batch. Prints the loss every tenth step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from hsdp_sharded_parameter_gb300.layers import TokenBlock  # noqa: E402


def train(steps=50, vocab=32000, hidden=1024, tokens=2048, rank_size=8, shard_size=4, dtype="bf16", p=0.1, lr=0.1, seed=1,
          say=print):
    """Runs `steps` steps; returns the losses."""
    block = TokenBlock(vocab, hidden, tokens, rank_size, shard_size, dtype=dtype, p=p, seed=seed)
    block.init_parameters(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    target = torch.randn(vocab, hidden, generator=gen, device="cuda").to(block.out[0].dtype)
    # the batch stays, so that a short run shows the loss fall
    ids = [torch.randint(0, vocab, (tokens,), generator=gen, device="cuda") for _ in range(rank_size)]
    losses = []
    for step in range(steps):
        out = block.forward(ids, step)
        diff = [o.float() - target[i].float() for o, i in zip(out, ids)]
        losses.append(torch.stack([d.square().mean() for d in diff]).mean())
        grad = [(d / tokens).to(out[0].dtype) for d in diff]
        block.backward(ids, grad, step)
        block.sgd(lr)
        if say and step % 10 == 0:
            say(f"step {step:4d}  loss {losses[-1].item():.4f}")
    block.close()
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    train(a.steps, a.vocab, a.hidden)
