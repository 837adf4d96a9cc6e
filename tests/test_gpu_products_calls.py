"""The products' calls as programs make them: several at once on streams of their
own, a process's first ones inside a capture, graphs that are replayed in turn,
views of larger tensors, one token, shards of one buffer."""
import os
import subprocess
import sys

import pytest
import torch

import products_ref as R
from hsdp_sharded_parameter_gb300 import capi as C
from test_gpu_products import BF16, Block, no_wait_ran_out, rand  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Steps:
    """The three operators in a row on operands and a workspace of their own."""

    def __init__(self, tokens, hidden, inner, seed):
        self.b = b = Block(tokens, hidden, inner, seed=seed)
        new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
        self.outs = [new(tokens, hidden), new(tokens, inner), new(tokens, inner), new(tokens, hidden), *(torch.empty_like(w) for w in b.w), new(inner, hidden)]
        self.work = torch.empty(max(C.fsdp_gated_ffn_workspace(tokens, hidden, inner), C.fsdp_gated_ffn_grad_workspace(tokens, hidden, inner),
                                    C.fsdp_orthogonalize_workspace(inner, hidden)), dtype=torch.uint8, device="cuda")

    def run(self):
        y, g, u, dx, dg, du, dd, o = self.outs
        C.fsdp_gated_ffn(self.b.x, *self.b.w, y, self.work, "silu", g, u)
        C.fsdp_gated_ffn_grad(self.b.grad, self.b.x, *self.b.w, g, u, dx, dg, du, dd, self.work)
        C.fsdp_orthogonalize(dg, o, self.work)

    def want(self):
        self.run()
        torch.cuda.synchronize()
        return [t.clone() for t in self.outs]


def same(steps, want):
    return all(torch.equal(a, b) for a, b in zip(steps.outs, want))


def test_streams_at_once():
    jobs = [Steps(300, 136, 520, 1), Steps(1, 512, 1376, 2), Steps(700, 264, 2056, 3), Steps(33, 64, 256, 4)]
    want = [j.want() for j in jobs]
    for j in jobs:
        for t in j.outs:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                j.run()
    torch.cuda.synchronize()
    assert all(same(j, w) for j, w in zip(jobs, want))


def test_graphs_in_turn():
    jobs = [Steps(300, 136, 520, 1), Steps(700, 264, 2056, 3)]
    want = [j.want() for j in jobs]
    graphs = []
    for j in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            j.run()
    for j in jobs:
        for t in j.outs:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(j, w) for j, w in zip(jobs, want))


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
from test_gpu_products_calls import Steps, same
from hsdp_sharded_parameter_gb300 import capi as C
job = Steps(300, 136, 520, 1)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    job.run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in job.outs]
assert same(job, job.want()) and all(torch.equal(a, b) for a, b in zip(got, job.outs))
assert C.fsdp_operators_status() == 0
print("equal")
"""


def test_a_process_may_begin_with_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


def test_views_of_one_buffer():
    # weights and their gradients as an unshard and a sync lay them out: one behind the other, from any element on
    t, h, f = 65, 72, 100
    sizes = [(f, h), (f, h), (h, f)]
    for offset in (0, 1, 8):
        flat, flat_grad = (torch.full((offset + 3 * f * h + 5,), 7.0, dtype=BF16, device="cuda") for _ in range(2))
        at = [offset + i * f * h for i in range(3)]
        w = [flat[a:a + f * h].view(s) for a, s in zip(at, sizes)]
        dw = [flat_grad[a:a + f * h].view(s) for a, s in zip(at, sizes)]
        for i, v in enumerate(w):
            v.copy_(rand(40 + i, *v.shape, 0.1))
        x, grad = rand(1, t, h), rand(2, t, h, 0.1)
        y, g, u, dx = torch.empty_like(x), torch.empty(t, f, dtype=BF16, device="cuda"), torch.empty(t, f, dtype=BF16, device="cuda"), torch.empty_like(x)
        work = torch.empty(C.fsdp_gated_ffn_grad_workspace(t, h, f, aligned=False), dtype=torch.uint8, device="cuda")
        C.fsdp_gated_ffn(x, *w, y, work, "gelu", g, u)
        R.agree("out", y, R.gated_ffn(x, *w, "gelu")["out"])
        C.fsdp_gated_ffn_grad(grad, x, *w, g, u, dx, *dw, work, "gelu")
        want = R.gated_ffn_grad(grad, x, *w, g, u, "gelu")
        for k, v in zip(("x", "w_gate", "w_up", "w_down"), [dx, *dw]):
            R.agree(k, v, want[k])
        assert bool((flat_grad[:offset] == 7).all()) and bool((flat_grad[offset + 3 * f * h:] == 7).all())


def test_batches_of_sequences():
    # (batch, sequence, hidden) as one matrix of tokens
    x, w = rand(1, 6, 64).view(2, 3, 64), [rand(2, 128, 64, 0.1), rand(3, 128, 64, 0.1), rand(4, 64, 128, 0.1)]
    y, g, u = torch.empty_like(x), torch.empty(2, 3, 128, dtype=BF16, device="cuda"), torch.empty(2, 3, 128, dtype=BF16, device="cuda")
    work = torch.empty(C.fsdp_gated_ffn_workspace(6, 64, 128), dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn(x, *w, y, work, gate=g, up=u)
    for k, v in R.gated_ffn(x.view(6, 64), *w, "silu").items():
        R.agree(k, {"out": y, "gate": g, "up": u}[k].view(6, -1), v)


def test_rows_that_overlap():
    # inputs of stride 0 (every row the same) and of rows that lie inside one another
    t, h, f = 70, 72, 136
    def over(seed, rows, cols, stride, std):  # noqa: E306
        return torch.as_strided(rand(seed, 1, (rows - 1) * stride + cols, std)[0], (rows, cols), (stride, 1))
    for stride in (0, 1, 8, 24):
        x, grad = over(1, t, h, stride, 1.0), over(2, t, h, stride, 0.1)
        w = [over(3, f, h, stride, 0.1), over(4, f, h, stride, 0.1), over(5, h, f, stride, 0.1)]
        g, u = over(6, t, f, stride, 1.0), over(7, t, f, stride, 1.0)
        y, dx, dw = torch.empty(t, h, dtype=BF16, device="cuda"), torch.empty(t, h, dtype=BF16, device="cuda"), [torch.empty(v.shape, dtype=BF16, device="cuda") for v in w]
        work = torch.empty(C.fsdp_gated_ffn_grad_workspace(t, h, f, aligned=False), dtype=torch.uint8, device="cuda")
        C.fsdp_gated_ffn(x, *w, y, work)
        R.agree("out", y, R.gated_ffn(x, *w, "silu")["out"])
        C.fsdp_gated_ffn_grad(grad, x, *w, g, u, dx, *dw, work)
        want = R.gated_ffn_grad(grad, x, *w, g, u, "silu")
        for k, v in zip(("x", "w_gate", "w_up", "w_down"), [dx, *dw]):
            R.agree(k, v, want[k])
        for rows, cols in [(40, 100), (100, 130)]:
            m = over(8, rows, cols, stride, 1.0)
            o = torch.empty(rows, cols, dtype=BF16, device="cuda")
            work = torch.empty(C.fsdp_orthogonalize_workspace(rows, cols), dtype=torch.uint8, device="cuda")
            C.fsdp_orthogonalize(m, o, work)
            assert R.distance(o, R.orthogonalize(m)) < 2.3e-3 + 5 * 2.0 ** -11


def test_the_longest_sums():
    # a sum of n random terms of size s wanders some 6 sqrt(n) s away from 0 at most; each of n / 16 additions
    # may cut 2^-21 of that, beside the terms' magnitudes' sum, 0.6 n s, (1 / 16) 2^-21 6 sqrt(n) / 0.6 = 2^-9.7
    n = 2 ** 24
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, grad, gate, up, w = r(n, 8), r(n, 8), r(n, 8), r(n, 8), [r(8, 8), r(8, 8), r(8, 8)]
    dx, dw = torch.empty_like(x), [torch.empty(8, 8, device="cuda") for _ in w]
    work = torch.empty(C.fsdp_gated_ffn_grad_workspace(n, 8, 8), dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn_grad(grad, x, *w, gate, up, dx, *dw, work, "relu")
    h = (gate.double().clamp(min=0) * up.double()).to(BF16).double()
    d = (grad.double() @ w[2].double())
    du, dg = (d * gate.double().clamp(min=0)).to(BF16).double(), (d * up.double() * (gate > 0)).to(BF16).double()
    for got, a, b in [(dw[0], dg, x.double()), (dw[1], du, x.double()), (dw[2], grad.double(), h)]:
        assert bool(((got.double() - a.T @ b).abs() <= 2.0 ** -9 * (a.abs().T @ b.abs())).all())
    y = torch.empty(3, 8, dtype=BF16, device="cuda")
    wide = [r(n, 8), r(n, 8), r(8, n)]
    work = torch.empty(C.fsdp_gated_ffn_workspace(3, 8, n), dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn(x[:3], *wide, y, work, "relu")
    h = ((x[:3].double() @ wide[0].double().T).clamp(min=0) * (x[:3].double() @ wide[1].double().T))
    # beside that h's rounding, 2^-8 of it
    assert bool(((y.double() - h @ wide[2].double().T).abs() <= (2.0 ** -9 + 2.0 ** -8) * (h.abs() @ wide[2].double().abs().T)).all())
