"""Trainable blocks on one HSDP unit, built from the training operators.

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


class GatedBlock:
    """The gated feed-forward block of a layer on one HSDP unit, with the
    optimizer step of its matrices: forward fsdp_gated_ffn on the gathered
    parameters, backward fsdp_gated_ffn_grad into the unit's gradients and
    their reduction, and an update by momentum that fsdp_orthogonalize makes
    orthogonal, of which every rank applies its own rows. The ranks live on one
    GPU, so each matrix's update is computed once."""

    def __init__(self, hidden, inner, tokens, rank_size, shard_size, activation="silu", device="cuda"):
        self.hidden, self.inner, self.activation = hidden, inner, activation
        # w_gate, w_up, w_down
        self.shapes = [(inner, hidden), (inner, hidden), (hidden, inner)]
        self.plan = C.Plan([s[0] for s in self.shapes], [s[1] for s in self.shapes], rank_size, shard_size).upload()
        self.unit = HsdpUnit(self.plan, "bf16", "bf16", device=device)
        new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        W = self.plan.W
        self.gate, self.up = ([new(tokens, inner) for _ in range(W)] for _ in range(2))
        self.out, self.grad_x = ([new(tokens, hidden) for _ in range(W)] for _ in range(2))
        self.momentum = [torch.zeros(s, dtype=torch.float32, device=device) for s in self.shapes]
        most = max(C.fsdp_gated_ffn_workspace(tokens, hidden, inner, aligned=False),
                   C.fsdp_gated_ffn_grad_workspace(tokens, hidden, inner, aligned=False),
                   C.fsdp_orthogonalize_workspace(inner, hidden), C.fsdp_orthogonalize_workspace(hidden, inner))
        self.work = new(most, dtype=torch.uint8)

    def init_parameters(self, seed=0, std=0.02):
        """The same N(0, std^2) values on every replica."""
        gen = torch.Generator(device=self.unit.device)
        gen.manual_seed(seed)
        for q, shape in enumerate(self.shapes):
            full = torch.randn(shape, generator=gen, device=self.unit.device) * std
            for w in range(self.plan.W):
                first, n = self.plan.sharded_size(q, w % self.plan.S)
                self.unit.shards[w * self.plan.P + q].copy_(full[first:first + n].reshape(-1))

    def _views(self, tensors, w):
        return [t.view(s) for t, s in zip(tensors[w * self.plan.P:(w + 1) * self.plan.P], self.shapes)]

    def forward(self, x):
        """x[w]: rank w's bfloat16 tokens. Returns out[w]."""
        self.unit.unshard_direct()
        for w in range(self.plan.W):
            C.fsdp_gated_ffn(x[w], *self._views(self.unit.full, w), self.out[w], self.work, self.activation, self.gate[w], self.up[w])
        return self.out

    def backward(self, x, grad_out, op="avg"):
        """grad_out[w]: the gradient of out[w]. Fills the unit's gradients,
        reduces them over the mesh and returns grad_x[w]."""
        for w in range(self.plan.W):
            C.fsdp_gated_ffn_grad(grad_out[w], x[w], *self._views(self.unit.full, w), self.gate[w], self.up[w], self.grad_x[w],
                                  *self._views(self.unit.grads, w), self.work, self.activation)
        self.unit.reduce_grads_one_pass(op)
        return self.grad_x

    def check_status(self):
        """Raises if a wait inside a kernel of the block's operators has run out
        since the last question: what they gave is undefined then. Synchronises
        the current stream."""
        if C.fsdp_operators_status():
            raise RuntimeError("gated block: a wait inside a kernel of its operators ran out")

    def step(self, lr, mu=0.95):
        """Momentum, orthogonalised, onto the shards: scaled by
        sqrt(max(1, rows / cols)). Asks check_status before the gradients go into
        the momentum and before an update goes onto the shards, but not while
        the stream is captured: a graph's user asks after the replay."""
        check = (lambda: None) if torch.cuda.is_current_stream_capturing() else self.check_status
        check()
        for q, (rows, cols) in enumerate(self.shapes):
            m = self.momentum[q].mul_(mu)
            spans = [self.plan.sharded_size(q, s) for s in range(self.plan.S)]
            for s, (first, n) in enumerate(spans):
                m[first:first + n].add_(self.unit.shard_grads[s * self.plan.P + q].view(n, cols))
            update = torch.empty(rows, cols, dtype=torch.bfloat16, device=m.device)
            C.fsdp_orthogonalize(m, update, self.work, scale=math.sqrt(max(1.0, rows / cols)))
            check()
            for w in range(self.plan.W):
                first, n = spans[w % self.plan.S]
                self.unit.shards[w * self.plan.P + q].view(n, cols).add_(update[first:first + n], alpha=-lr)

    def close(self):
        self.unit.close()
        self.plan.close()
