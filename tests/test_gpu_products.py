"""The gated feed-forward block, its gradient and the orthogonalised update on
the GPU against their definitions in 64 bits (products_ref). Each output lies
inside a larger buffer of a known pattern, and nothing outside it, nor behind a
workspace, may change."""
import math

import pytest
import torch

import products_ref as R
from hsdp_sharded_parameter_gb300 import capi as C
from test_gpu_operators import Guarded, Workspace

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert C.fsdp_operators_status() == 0


def rand(seed, rows, cols, std=1.0, dtype=BF16, pad=0, offset=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = Guarded(rows, cols, dtype, pad, offset).t
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std + 0.05 * std)
    return x


def on_grid(*tensors):
    return all(t.data_ptr() % 16 == 0 and t.stride(0) % 8 == 0 and t.stride(0) >= t.shape[1] for t in tensors if t is not None)


class Block:
    """A block's operands at these sizes; pad and offset (elements) apply to all of them."""

    def __init__(self, tokens, hidden, inner, pad=0, offset=0, seed=1):
        self.sizes, self.pad, self.offset = (tokens, hidden, inner), pad, offset
        k = lambda i, r, c, std: rand(seed * 100 + i, r, c, std, BF16, pad, offset)  # noqa: E731
        self.x = k(0, tokens, hidden, 1.0)
        self.w = [k(1, inner, hidden, hidden ** -0.5 if hidden else 1.0), k(2, inner, hidden, hidden ** -0.5 if hidden else 1.0),
                  k(3, hidden, inner, inner ** -0.5 if inner else 1.0)]
        self.gate, self.up, self.grad = k(4, tokens, inner, 1.0), k(5, tokens, inner, 1.0), k(6, tokens, hidden, 0.1)

    def out(self, rows, cols, dtype=BF16):
        return Guarded(rows, cols, dtype, self.pad, self.offset)

    def forward(self, act="silu", keep=True, stream=None):
        t, h, f = self.sizes
        y, g, u = self.out(t, h), self.out(t, f), self.out(t, f)
        work = Workspace(C.fsdp_gated_ffn_workspace(t, h, f, aligned=on_grid(self.x, *self.w)))
        C.fsdp_gated_ffn(self.x, *self.w, y.t, work.t, act, g.t if keep else None, u.t if keep else None, stream=stream)
        torch.cuda.synchronize()
        work.check()
        return {"out": y.check(), "gate": g.check(), "up": u.check()} if keep else {"out": y.check()}

    def backward(self, act="silu", dtype=BF16, before=None):
        t, h, f = self.sizes
        outs = {"x": self.out(t, h), "w_gate": self.out(f, h, dtype), "w_up": self.out(f, h, dtype), "w_down": self.out(h, f, dtype)}
        for k, v in (before or {}).items():
            outs[k].t.copy_(v)
        work = Workspace(C.fsdp_gated_ffn_grad_workspace(t, h, f, aligned=on_grid(self.x, self.grad, *self.w)))
        C.fsdp_gated_ffn_grad(self.grad, self.x, *self.w, self.gate, self.up, *(o.t for o in outs.values()), work.t, act,
                              accumulate=before is not None)
        torch.cuda.synchronize()
        work.check()
        return {k: o.check() for k, o in outs.items()}


SIZES = [(1, 8, 8), (1, 1, 1), (2, 64, 128), (1, 512, 1376), (3, 17, 5), (16, 256, 704), (33, 130, 257), (128, 128, 128), (129, 136, 264),
         (200, 72, 1000), (257, 511, 300), (300, 1024, 512), (512, 320, 864), (700, 264, 2056)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("pad, offset", [(0, 0), (3, 1), (8, 8)])
def test_gated_ffn(sizes, pad, offset):
    b = Block(*sizes, pad=pad, offset=offset)
    want = R.gated_ffn(b.x, *b.w, "silu")
    for keep in (True, False):
        for k, v in b.forward("silu", keep).items():
            R.agree(k, v, want[k])
    assert R.distance(v, want["out"][0]) < 5e-3


@pytest.mark.parametrize("act", ["gelu", "relu"])
@pytest.mark.parametrize("sizes", [(5, 40, 24), (140, 96, 300)], ids=str)
def test_activations(act, sizes):
    b = Block(*sizes)
    want = R.gated_ffn(b.x, *b.w, act)
    for k, v in b.forward(act).items():
        R.agree(k, v, want[k])
    want = R.gated_ffn_grad(b.grad, b.x, *b.w, b.gate, b.up, act)
    for k, v in b.backward(act).items():
        R.agree(k, v, want[k])


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("pad, offset", [(0, 0), (3, 1), (8, 8)])
def test_gated_ffn_grad(sizes, pad, offset):
    b = Block(*sizes, pad=pad, offset=offset)
    want = R.gated_ffn_grad(b.grad, b.x, *b.w, b.gate, b.up, "silu")
    for k, v in b.backward().items():
        R.agree(k, v, want[k])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 3])
def test_gradients_accumulate(dtype, pad):
    b = Block(150, 72, 136, pad=pad)
    t, h, f = b.sizes
    before = {"w_gate": rand(7, f, h, 0.5, dtype), "w_up": rand(8, f, h, 0.5, dtype), "w_down": rand(9, h, f, 0.5, dtype)}
    want = R.gated_ffn_grad(b.grad, b.x, *b.w, b.gate, b.up, "silu", dtype, before)
    for k, v in b.backward(dtype=dtype, before=before).items():
        R.agree(k, v, want[k])
    want = R.gated_ffn_grad(b.grad, b.x, *b.w, b.gate, b.up, "silu", dtype)
    for k, v in b.backward(dtype=dtype).items():
        R.agree(k, v, want[k])


@pytest.mark.parametrize("sizes", [(0, 64, 72), (5, 0, 16), (5, 16, 0), (0, 0, 0), (130, 0, 136), (130, 136, 0)], ids=str)
def test_sums_over_nothing(sizes):
    b = Block(*sizes)
    for k, v in b.forward("silu", True).items():
        assert not bool(v.any()), k
    before = {k: torch.ones_like(w) for k, w in zip(("w_gate", "w_up", "w_down"), b.w)}
    for k, v in b.backward(before=before).items():
        assert bool((v == (0 if k == "x" else 1)).all()), k
    for k, v in b.backward().items():
        assert not bool(v.any()), k


def matrix(kind, rows, cols, dtype, pad=0, offset=0, std=1e-3, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64)
    if kind != "noise":
        k = min(rows, cols, 8)
        s = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.float64) @ torch.randn(k, cols, generator=g, device="cuda", dtype=torch.float64)
        x = s + {"spikes": 0.1, "low": 0.001}[kind] * x
    out = Guarded(rows, cols, dtype, pad, offset).t
    out.copy_(x * std)
    return out


def ortho(x, pad=0, offset=0, **k):
    rows, cols = x.shape
    out = Guarded(rows, cols, BF16, pad, offset)
    work = Workspace(C.fsdp_orthogonalize_workspace(rows, cols))
    C.fsdp_orthogonalize(x, out.t, work.t, **k)
    torch.cuda.synchronize()
    work.check()
    return out.check()


# Rounding the result is off by at most 2^-8, in the 2-norm by that over the
# square root of 3: 2.3e-3. A step's roundings to binary16 (the factors of its
# product, A and the polynomial), 2^-12 over the square root of 3 each, four of
# them, reach the result with a weight of the order of one: 2^-11 a step, 2.4e-3
# for five.
ORTHO = 5e-3
MATRICES = [(64, 200), (65, 200), (300, 65), (63, 5000), (5000, 2), (1, 1), (1, 100), (37, 1), (8, 8), (16, 64), (64, 16), (100, 100), (128, 384), (129, 257), (300, 200), (256, 256), (511, 777),
            (1000, 1000), (640, 320), (1030, 520), (520, 1290)]


@pytest.mark.parametrize("rows, cols", MATRICES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["noise", "spikes"])
def test_orthogonalize(rows, cols, dtype, kind):
    x = matrix(kind, rows, cols, dtype)
    assert R.distance(ortho(x), R.orthogonalize(x)) < ORTHO


@pytest.mark.parametrize("rows, cols", [(64, 130), (300, 300)])
@pytest.mark.parametrize("kind", ["spikes", "low"])
@pytest.mark.parametrize("std", [1e-30, 1e-12, 1.0, 1e12, 1e30])
def test_orthogonalize_any_size_of_values(rows, cols, kind, std):
    x = matrix(kind, rows, cols, F32, std=std)
    assert R.distance(ortho(x, eps=0.0), R.orthogonalize(x, eps=0.0)) < ORTHO


@pytest.mark.parametrize("pad, offset", [(3, 1), (8, 8), (1, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(50, 131), (131, 50)])
def test_orthogonalize_strides(rows, cols, dtype, pad, offset):
    x = matrix("spikes", rows, cols, dtype, pad, offset)
    assert R.distance(ortho(x, pad, offset, scale=0.25), R.orthogonalize(x, scale=0.25)) < ORTHO


@pytest.mark.parametrize("steps, coefficients", [(1, (3.4445, -4.7750, 2.0315)), (3, (3.4445, -4.7750, 2.0315)), (6, (3.4445, -4.7750, 2.0315)),
                                                 (12, (1.875, -1.25, 0.375)), (5, (2.0, -1.5, 0.5)), (4, (1.5, -0.5, 0.0))])
def test_orthogonalize_other_polynomials(steps, coefficients):
    for rows, cols in [(96, 200), (200, 96)]:
        x = matrix("noise", rows, cols, F32)
        want = R.orthogonalize(x, steps, coefficients)
        assert R.distance(ortho(x, steps=steps, coefficients=coefficients), want) < 2.3e-3 + 2.0 ** -11 * steps + 1e-4


def test_orthogonalize_borders():
    assert not bool(ortho(torch.zeros(40, 70, device="cuda")).any())
    for bad in (math.inf, math.nan):
        x = matrix("noise", 40, 70, F32).clone()
        x[3, 5] = bad
        assert bool(torch.isnan(ortho(x)).all())
    for shape in [(0, 5), (5, 0), (0, 0)]:
        ortho(torch.zeros(*shape, device="cuda"))


def test_equal_bits_on_other_streams_and_in_graphs():
    # one graph of the three operators in a row, one workspace
    b = Block(300, 136, 520)
    t, h, f = b.sizes
    new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    y, g, u, dx, d = new(t, h), new(t, f), new(t, f), new(t, h), [torch.empty_like(w) for w in b.w]
    o = new(f, h)
    work = torch.empty(max(C.fsdp_gated_ffn_workspace(t, h, f), C.fsdp_gated_ffn_grad_workspace(t, h, f), C.fsdp_orthogonalize_workspace(f, h)),
                       dtype=torch.uint8, device="cuda")

    def run():
        C.fsdp_gated_ffn(b.x, *b.w, y, work, "silu", g, u)
        C.fsdp_gated_ffn_grad(b.grad, b.x, *b.w, g, u, dx, *d, work)
        C.fsdp_orthogonalize(d[0], o, work)

    run()
    torch.cuda.synchronize()
    outs = [y, g, u, dx, *d, o]
    want = [v.clone() for v in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, v) for a, v in zip(outs, want))
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, v) for a, v in zip(outs, want))


def test_gated_block_on_a_mesh():
    from hsdp_sharded_parameter_gb300.layers import GatedBlock

    block = GatedBlock(72, 200, 90, 4, 2)
    block.init_parameters(1, 0.1)
    x, grad = [rand(10 + w, 90, 72) for w in range(4)], [rand(20 + w, 90, 72, 0.1) for w in range(4)]
    out = block.forward(x)
    grad_x = block.backward(x, grad)
    mean = [0.0, 0.0, 0.0]
    for w in range(4):
        p = block._views(block.unit.full, w)
        R.agree("out", out[w], R.gated_ffn(x[w], *p, "silu")["out"])
        want = R.gated_ffn_grad(grad[w], x[w], *p, block.gate[w], block.up[w], "silu")
        R.agree("grad_x", grad_x[w], want["x"])
        for q, k in enumerate(("w_gate", "w_up", "w_down")):
            R.agree(k, block._views(block.unit.grads, w)[q], want[k])
            mean[q] = mean[q] + R.d(block._views(block.unit.grads, w)[q]) / 4
    before = [t.clone() for t in block.unit.shards]
    block.step(0.5)
    for q, (rows, cols) in enumerate(block.shapes):
        # the reduced gradient is rounded to bfloat16, which the update sees as 2^-8 of its values at most
        got = torch.cat([block.unit.shard_grads[s * 3 + q].view(-1, cols) for s in range(2)])
        assert bool(((R.d(got) - mean[q]).abs() <= 2.0 ** -8 * mean[q].abs() + 1e-6).all())
        update = R.orthogonalize(got, scale=max(1.0, rows / cols) ** 0.5)
        for w in range(4):
            first, n = block.plan.sharded_size(q, w % 2)
            moved = R.d(before[w * 3 + q]).view(n, cols) - R.d(block.unit.shards[w * 3 + q]).view(n, cols)
            # each value is rounded once more as it is added: by 2^-8 of what it becomes
            off = (moved - 0.5 * update[first:first + n]).norm()
            assert float(off) <= ORTHO * 0.5 * float(update.norm()) + 2.0 ** -8 * float(R.d(block.unit.shards[w * 3 + q]).norm())
    block.close()
