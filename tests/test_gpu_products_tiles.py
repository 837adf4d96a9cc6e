"""The products at sizes at which every pair of SMs computes several tiles: the
tensor memory's halves are handed over again and again, the ring runs on from
tile to tile, and tiles of both widths have all their epilogues. Sizes are odd or
off the tiles' grid; bounds are products_ref's and test_gpu_orthogonalize's."""
import pytest
import torch

import products_ref as R
from hsdp_sharded_parameter_gb300 import capi as C
from test_gpu_orthogonalize import DEFAULT, ROUNDED
from test_gpu_products import BF16, F32, Block, matrix, no_wait_ran_out, ortho, rand  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, hidden, inner: many tiles of (tokens x inner), of (tokens x hidden), of the weights' gradients
MANY = {"inner": (4801, 200, 4004), "inner, slim": (5001, 200, 4101), "hidden": (4801, 4004, 200), "hidden, slim": (5001, 4101, 200),
        "weights": (130, 2600, 2609), "weights, slim": (130, 2500, 2505)}


@pytest.mark.parametrize("which", ["inner", "inner, slim", "hidden", "hidden, slim"])
@pytest.mark.parametrize("pad, offset", [(0, 0), (3, 1)])
def test_gated_ffn(which, pad, offset):
    b = Block(*MANY[which], pad=pad, offset=offset)
    want = R.gated_ffn(b.x, *b.w, "silu")
    for keep in (True, False):
        for k, v in b.forward("silu", keep).items():
            R.agree(k, v, want[k])


@pytest.mark.parametrize("which", list(MANY))
@pytest.mark.parametrize("dtype, accumulate, pad, offset", [(BF16, False, 0, 0), (F32, True, 0, 0), (BF16, True, 3, 1), (F32, False, 8, 8)])
def test_gated_ffn_grad(which, dtype, accumulate, pad, offset):
    b = Block(*MANY[which], pad=pad, offset=offset)
    t, h, f = b.sizes
    before = {"w_gate": rand(7, f, h, 0.5, dtype), "w_up": rand(8, f, h, 0.5, dtype), "w_down": rand(9, h, f, 0.5, dtype)} if accumulate else None
    want = R.gated_ffn_grad(b.grad, b.x, *b.w, b.gate, b.up, "silu", dtype, before)
    for k, v in b.backward(dtype=dtype, before=before).items():
        R.agree(k, v, want[k])


def orthogonalize(x, steps, coefficients):
    """As products_ref's, where x is."""
    a, b, c = coefficients
    x = x.double()
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(steps):
        g = x @ x.mT if x.shape[0] <= x.shape[1] else x.mT @ x
        m = b * g + c * g @ g
        x = a * x + (m @ x if x.shape[0] <= x.shape[1] else x @ m)
    return x


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


MATRICES = {"wide": (6100, 6151), "tall": (6151, 6100), "slim": (5001, 4351), "one tile a pair": (2701, 2803), "one tile a pair, tall": (2803, 2701)}


@pytest.mark.parametrize("which, steps, dtype, pad, offset", [("wide", 2, F32, 0, 0), ("tall", 2, BF16, 0, 0), ("slim", 2, F32, 3, 1), ("one tile a pair", 5, BF16, 3, 1),
                                                              ("one tile a pair, tall", 5, F32, 1, 0)])
def test_orthogonalize(which, steps, dtype, pad, offset):
    x = matrix("spikes", *MATRICES[which], dtype, pad, offset)
    assert off(ortho(x, pad, offset, steps=steps), orthogonalize(x, steps, DEFAULT)) < ROUNDED + steps * 2.0 ** -11


@pytest.mark.parametrize("pad, offset", [(3, 1), (8, 8), (1, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(150, 331), (331, 150)])
def test_orthogonalize_strides(rows, cols, dtype, pad, offset):
    x = matrix("spikes", rows, cols, dtype, pad, offset)
    assert R.distance(ortho(x, pad, offset, scale=0.25), R.orthogonalize(x, scale=0.25)) < ROUNDED + 5 * 2.0 ** -11


@pytest.mark.parametrize("rows, cols", [(100, 130), (300, 300), (130, 100)])
@pytest.mark.parametrize("steps", [8, 12])
def test_orthogonalize_more_steps(rows, cols, steps):
    x = matrix("noise", rows, cols, F32)
    assert R.distance(ortho(x, steps=steps), R.orthogonalize(x, steps)) < ROUNDED + steps * 2.0 ** -11


def kernels(call):
    """(width, epilogue) of the products that a call runs."""
    from torch.profiler import ProfilerActivity, profile

    call()
    for _ in range(3):  # a process's first record may be empty
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        names = [e.key for e in p.key_averages() if "product_kernel<" in e.key]
        if names:
            break
    else:
        pytest.skip("the profiler records no kernels here")
    found = set()
    for n in names:
        width, epilogue = n.split("product_kernel<")[1].split(">(")[0].split(", ", 1)
        found.add((int(width), epilogue.split("::")[-1].split("<")[0]))
    return found


def test_the_sizes_have_the_tiles_they_are_for():
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2

    def check(found, width, epilogue, tiles, least=4):
        assert (width, epilogue) in found, (width, epilogue, found)
        assert tiles >= least * pairs - 8, (tiles, pairs)

    up = lambda n, by: -(-n // by)  # noqa: E731
    for which, (t, h, f) in MANY.items():
        b = Block(t, h, f)
        forward, backward, w = kernels(lambda: b.forward("silu", True)), kernels(b.backward), 128 if "slim" in which else 256
        if "inner" in which:
            # (gate and up side by side take half of a tile's columns each)
            check(forward, 256, "Gated", up(t, 256) * up(f, 128))
            check(backward, w, "GatedGrad", up(t, 256) * up(f, w))
        elif "hidden" in which:
            check(forward, w, "Store", up(t, 256) * up(h, w))
            check(backward, w, "Store", up(t, 256) * up(h, w))
        else:
            check(backward, w, "Store", 3 * up(f, 256) * up(h, w))
    for which, (m, n) in MATRICES.items():
        x = matrix("noise", m, n, F32)
        found, w, p = kernels(lambda: ortho(x, steps=1)), 128 if which == "slim" else 256, up(min(m, n), 256)
        least = 4 if "one" not in which else 0
        for epilogue in ("Gram", "Poly"):
            check(found, w, epilogue, p * (p + 1) // 2 * (256 // w), least)
        check(found, w, "Next", up(m, 256) * up(n, w), least)
