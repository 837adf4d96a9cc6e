"""A trainable block on one HSDP unit, built from the training operators.

``TokenBlock`` is the input end of a pre-norm transformer with one sublayer,
for all rank_size virtual ranks of a plan. Its parameters are sharded with the
unit's plan, gathered by ``unshard_direct`` and their gradients, which the
operators write straight into the unit's buffers, reduced by
``reduce_grads_one_pass``:

    e = scale * table[ids]                   fsdp_embedding
    h = drop(e);  n = norm(h)                fsdp_layer_norm
    y = n @ linear^T                         a library matrix product
    out = h + drop(y)                        fsdp_dropout

and backwards fsdp_dropout on the gradient of out, the two products of the
linear layer, fsdp_layer_norm_grad (which takes the residual stream's gradient
along) and fsdp_embedding_grad. Masks are drawn from (seed, draw), a draw of
its own for every step, rank and place, so the backward pass makes them again
and nothing stores them.
"""
from __future__ import annotations

import math

import torch

from . import capi as C
from .runtime import TORCH_DT, HsdpUnit


class TokenBlock:
    def __init__(self, vocab, hidden, tokens, rank_size, shard_size, dtype="bf16", p=0.1, eps=1e-5, seed=0,
                 device="cuda"):
        """Buffers for `tokens` tokens a rank; the workspaces are shared by the
        ranks, whose calls follow each other on one stream."""
        self.vocab, self.hidden, self.tokens = vocab, hidden, tokens
        self.p, self.eps, self.seed, self.scale = float(p), float(eps), int(seed), math.sqrt(hidden)
        # table, norm weight, norm bias, linear layer
        self.plan = C.Plan([vocab, hidden, hidden, hidden], [hidden, 1, 1, hidden], rank_size, shard_size).upload()
        self.unit = HsdpUnit(self.plan, dtype, dtype, device=device)
        dt, W = TORCH_DT[dtype], self.plan.W
        new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device=device)  # noqa: E731
        rows = lambda: [new(tokens, hidden) for _ in range(W)]  # noqa: E731
        self.h, self.n, self.y, self.out = rows(), rows(), rows(), rows()
        self.mean, self.rstd = ([new(tokens, dtype=torch.float32) for _ in range(W)] for _ in range(2))
        self.scratch = [new(tokens, hidden) for _ in range(2)]
        self.emb_work = new(C.fsdp_embedding_grad_workspace(tokens, vocab, hidden), dtype=torch.uint8)
        self.norm_work = new(C.fsdp_layer_norm_grad_workspace(tokens, hidden), dtype=torch.uint8)

    def init_parameters(self, seed=0, std=0.02):
        """The same values on every replica: table and linear N(0, std^2),
        weight 1, bias 0. (A shard is cut from the full parameter by the plan's
        own offsets.)"""
        gen = torch.Generator(device=self.unit.device)
        gen.manual_seed(seed)
        H, dev = self.hidden, self.unit.device
        full = [torch.randn(self.vocab, H, generator=gen, device=dev) * std, torch.ones(H, device=dev),
                torch.zeros(H, device=dev), torch.randn(H, H, generator=gen, device=dev) * std]
        for w in range(self.plan.W):
            for q in range(self.plan.P):
                first, n = self.plan.sharded_size(q, w % self.plan.S)
                self.unit.shards[w * self.plan.P + q].copy_(full[q][first:first + n].reshape(-1))

    def _views(self, tensors, w):
        t = tensors[w * self.plan.P:(w + 1) * self.plan.P]
        return t[0].view(self.vocab, self.hidden), t[1], t[2], t[3].view(self.hidden, self.hidden)

    def _draws(self, step, w):
        """The draws of a rank's two dropouts in a step."""
        return (2 * (step * self.plan.W + w)) & 0xFFFFFFFF, (2 * (step * self.plan.W + w) + 1) & 0xFFFFFFFF

    def forward(self, ids, step=0):
        """ids[w]: rank w's int32 or int64 token ids (those outside the
        vocabulary are padding). Returns out[w], the ranks' residual streams."""
        self.unit.unshard_direct()
        for w in range(self.plan.W):
            table, weight, bias, linear = self._views(self.unit.full, w)
            d0, d1 = self._draws(step, w)
            emb = self.scratch[0]
            C.fsdp_embedding(table, ids[w], emb, scale=self.scale)
            C.fsdp_layer_norm(emb, weight, bias, self.n[w], self.mean[w], self.rstd[w], eps=self.eps, hidden=self.h[w],
                              p=self.p, seed=self.seed, draw=d0)
            torch.matmul(self.n[w], linear.t(), out=self.y[w])
            C.fsdp_dropout(self.y[w], self.out[w], self.p, self.seed, d1, residual=self.h[w])
        return self.out

    def backward(self, ids, grad_out, step=0, op="avg"):
        """grad_out[w]: the gradient of out[w]. Fills the unit's gradients and
        reduces them over the mesh into unit.shard_grads."""
        grad_y, grad_n = self.scratch
        for w in range(self.plan.W):
            _, weight, _, linear = self._views(self.unit.full, w)
            g_table, g_weight, g_bias, g_linear = self._views(self.unit.grads, w)
            d0, d1 = self._draws(step, w)
            C.fsdp_dropout(grad_out[w], grad_y, self.p, self.seed, d1)
            torch.matmul(grad_y.t(), self.n[w], out=g_linear)
            torch.matmul(grad_y, linear, out=grad_n)
            grad_e = grad_y  # its last use is behind us
            C.fsdp_layer_norm_grad(grad_n, self.h[w], self.mean[w], self.rstd[w], weight, grad_e, g_weight, g_bias,
                                   self.norm_work, grad_hidden=grad_out[w], p=self.p, seed=self.seed, draw=d0)
            C.fsdp_embedding_grad(grad_e, ids[w], g_table, self.emb_work, scale=self.scale)
        self.unit.reduce_grads_one_pass(op)

    def sgd(self, lr):
        """Plain gradient descent on the shards."""
        for shard, grad in zip(self.unit.shards, self.unit.shard_grads):
            shard.add_(grad, alpha=-lr)

    def close(self):
        self.unit.close()
        self.plan.close()
