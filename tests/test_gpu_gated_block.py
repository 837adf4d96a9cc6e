"""layers.GatedBlock beside what test_gpu_products holds of it: a wait that ran
out, and a whole step in a graph. The wait is a status that the test gives, not
one of the GPU's."""
import pytest
import torch

from hsdp_sharded_parameter_gb300 import capi as C
from hsdp_sharded_parameter_gb300.layers import GatedBlock
from test_gpu_products import rand

pytestmark = pytest.mark.gpu


def make():
    block = GatedBlock(72, 200, 90, 4, 2)
    block.init_parameters(1, 0.1)
    return block, [rand(10 + w, 90, 72) for w in range(4)], [rand(20 + w, 90, 72, 0.1) for w in range(4)]


@pytest.mark.parametrize("asked", [1, 2, 4])
def test_no_step_from_undefined_results(monkeypatch, asked):
    block, x, grad = make()
    block.forward(x)
    block.backward(x, grad)
    before, momentum = [t.clone() for t in block.unit.shards], [t.clone() for t in block.momentum]
    calls = []
    monkeypatch.setattr(C, "fsdp_operators_status", lambda stream=None: int(calls.append(0) is None and len(calls) == asked))
    with pytest.raises(RuntimeError, match="ran out"):
        block.step(0.5)
    # the question before the momentum, and one before each matrix's shards move
    for q in range(3):
        moved = [not torch.equal(before[w * 3 + q], block.unit.shards[w * 3 + q]) for w in range(4)]
        assert all(moved) if q < asked - 2 else not any(moved)
    if asked == 1:
        assert all(torch.equal(a, b) for a, b in zip(momentum, block.momentum))
    block.close()


def test_a_training_step_in_a_graph():
    block, x, grad = make()
    start = [t.clone() for t in block.unit.shards]

    def run():
        block.forward(x)
        block.backward(x, grad)
        block.step(0.05)

    run()
    run()
    want = [t.clone() for t in block.unit.shards]
    for t, s in zip(block.unit.shards, start):
        t.copy_(s)
    for m in block.momentum:
        m.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(block.unit.shards, want))
    block.check_status()
    block.close()
