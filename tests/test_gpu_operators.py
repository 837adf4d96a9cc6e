"""The training operators on the GPU against their definitions in 64 bits
(operators_ref): values, types, alignments, strides, odd sizes, empty rows,
infinities and NaN in dropped places, equal bits on equal calls, graphs and
side streams. Each output lies inside a larger buffer of a known pattern, and
nothing outside it may change. Errors are bounded value by value; the bounds
are derived in operators_ref."""
import itertools
import math

import numpy as np
import pytest
import torch

import operators_ref as R
from hsdp_sharded_parameter_gb300 import capi as C

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = {"f32": F32, "bf16": BF16}


class Guarded:
    """A rows x cols matrix at an element offset and row stride inside a
    buffer of 0x5A bytes; check() finds every change outside the matrix."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0):
        self.shape = (rows, cols)
        self.stride = cols + pad
        n = offset + max(rows, 1) * self.stride + 64
        self.buf = torch.empty(n, dtype=dtype, device="cuda")
        self.buf.view(torch.uint8).fill_(0x5A)
        self.t = torch.as_strided(self.buf, (rows, cols), (self.stride, 1), offset)
        self.offset = offset

    def check(self):
        b = self.buf.clone()
        torch.as_strided(b, self.shape, (self.stride, 1), self.offset).copy_(torch.as_strided(
            torch.empty_like(b).view(torch.uint8).fill_(0x5A).view(b.dtype), self.shape, (self.stride, 1), self.offset))
        assert bool((b.view(torch.uint8) == 0x5A).all()), "bytes outside an output changed"
        return self.t


class Workspace:
    """A workspace of exactly the bytes asked for, followed by a known pattern."""

    def __init__(self, nbytes):
        self.buf = torch.full((nbytes + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        self.t = self.buf[:nbytes]

    def check(self):
        assert bool((self.buf[self.t.numel():] == 0x5A).all()), "bytes behind the workspace changed"


def rand(seed, rows, cols, dtype, std=1.0, pad=0, offset=0, shift=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = Guarded(rows, cols, dtype, pad, offset).t
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std + shift)
    return x


def vec(seed, n, dtype, shift=0.0):
    return rand(seed, 1, n, dtype, shift=shift).reshape(n)


def ids_of(seed, n, vocab, kind, dtype=torch.int64):
    g = torch.Generator()
    g.manual_seed(seed)
    ids = torch.randint(0, max(vocab, 1), (n,), generator=g)
    if kind == "hot":
        ids = torch.where(torch.rand(n, generator=g) < 0.9, ids % 3 % max(vocab, 1), ids)
    elif kind == "one":
        ids[:] = vocab - 1
    elif kind == "none":
        ids[:] = -1
    elif kind == "wild":  # ids that name no row, far and near
        wild = torch.tensor([-1, vocab, vocab + 1, -(2 ** 31), 2 ** 31 - 1])
        ids = torch.where(torch.rand(n, generator=g) < 0.4, wild[torch.randint(0, 5, (n,), generator=g)], ids)
    elif kind == "sorted":
        ids = ids.sort().values
    return ids.to(dtype).cuda()


# --------------------------------------------------------------- embedding

@pytest.mark.parametrize("tdt, odt", list(itertools.product(NAMES, NAMES)))
@pytest.mark.parametrize("n, vocab, cols, pad, offset", [
    (1, 1, 1, 0, 0), (3, 7, 8, 0, 0), (17, 5, 264, 0, 0), (33, 100, 257, 0, 0), (9, 11, 1111, 3, 1), (5, 40, 512, 8, 0),
    (64, 9, 31, 0, 5), (2, 3, 4104, 0, 0)])
def test_embedding(tdt, odt, n, vocab, cols, pad, offset):
    table = rand(1, vocab, cols, NAMES[tdt], 0.02, pad, offset)
    ids = ids_of(2, n, vocab, "wild", torch.int64 if n % 2 else torch.int32)
    out = Guarded(n, cols, NAMES[odt], pad, (offset * 3) % 8)
    C.fsdp_embedding(table, ids, out.t, scale=math.sqrt(cols))
    R.agree("out", out.check(), R.embedding(table, ids, math.sqrt(cols), 0, NAMES[odt]))


# more than one block of the narrow kernel (1024 granules), on the grid and off it, and of the wide one, in one and in several steps a row
MANY_TOKENS = [(1500, 300, 8, 0, 0), (1030, 77, 40, 0, 0), (700, 50, 93, 0, 1), (700, 50, 200, 0, 0), (500, 40, 201, 3, 0), (300, 90, 520, 0, 0),
               (150, 33, 1111, 0, 3), (70, 20, 4104, 0, 0), (65, 20, 4999, 1, 0)]


@pytest.mark.parametrize("tdt, odt", list(itertools.product(NAMES, NAMES)))
@pytest.mark.parametrize("n, vocab, cols, pad, offset", MANY_TOKENS)
def test_embedding_of_many_tokens(tdt, odt, n, vocab, cols, pad, offset):
    table = rand(1, vocab, cols, NAMES[tdt], 0.02, pad, offset)
    ids = ids_of(2, n, vocab, "wild", torch.int32 if n % 2 else torch.int64)
    out = Guarded(n, cols, NAMES[odt], pad, (offset * 3) % 8)
    C.fsdp_embedding(table, ids, out.t, scale=0.7)
    R.agree("out", out.check(), R.embedding(table, ids, 0.7, 0, NAMES[odt]))


def test_embedding_ids_beyond_32_bits_and_a_slice_of_the_vocabulary():
    table = rand(1, 10, 40, BF16)
    ids = torch.tensor([2 ** 32 + 3, 2 ** 40, -(2 ** 63), 2 ** 63 - 1, 100, 109, 110, 99, 3], device="cuda")
    for first in (0, 100, 2 ** 32, -5):
        out = Guarded(len(ids), 40, BF16)
        C.fsdp_embedding(table, ids, out.t, first_row=first)
        R.agree("out", out.check(), R.embedding(table, ids, 1.0, first, BF16))
        part, whole = (torch.zeros(10, 40, device="cuda") for _ in range(2))
        grad = rand(3, len(ids), 40, F32)
        w = torch.empty(C.fsdp_embedding_grad_workspace(len(ids), 10, 40), dtype=torch.uint8, device="cuda")
        C.fsdp_embedding_grad(grad, ids, part, w, first_row=first)
        R.agree("grad", part, R.embedding_grad(grad, ids, 10, 1.0, first, F32))


def test_embedding_of_no_tokens_no_rows_and_unnamed_infinities():
    table = torch.full((4, 24), float("inf"), dtype=BF16, device="cuda")
    ids = torch.tensor([[-1, 7], [4, -9]], device="cuda")
    out = Guarded(4, 24, F32)
    C.fsdp_embedding(table, ids, out.t)
    assert bool((out.check() == 0).all())
    C.fsdp_embedding(table, ids[:0], out.t[:0])
    C.fsdp_embedding(table[:0], ids, out.t)
    assert bool((out.check() == 0).all())


GRAD_KINDS = ["uniform", "hot", "one", "none", "wild", "sorted"]


@pytest.mark.parametrize("kind", GRAD_KINDS)
@pytest.mark.parametrize("n, vocab, cols, gdt, tdt", [
    (1, 1, 1, "f32", "f32"), (31, 4, 8, "bf16", "bf16"), (32, 50, 256, "bf16", "f32"), (33, 300, 257, "f32", "bf16"),
    (300, 4099, 67, "f32", "f32"), (1025, 70, 130, "bf16", "bf16"), (2100, 256, 264, "bf16", "f32"), (700, 65535, 9, "f32", "f32"),
    (5000, 3, 40, "f32", "f32"), (300, 50, 1300, "bf16", "f32"), (512, 64, 513, "f32", "f32"), (513, 70, 1300, "f32", "bf16"),
    (512, 63, 24, "bf16", "bf16")])
def test_embedding_grad(kind, n, vocab, cols, gdt, tdt):
    grad = rand(4, n, cols, NAMES[gdt], pad=(3 if cols % 2 else 8) * (n % 2))
    ids = ids_of(5, n, vocab, kind, torch.int32 if n % 2 else torch.int64)
    out = Guarded(vocab, cols, NAMES[tdt], 5 * (cols % 2), cols % 2)
    work = Workspace(C.fsdp_embedding_grad_workspace(n, vocab, cols))
    w = work.t
    C.fsdp_embedding_grad(grad, ids, out.t, w, scale=0.7)
    R.agree("grad", out.check(), R.embedding_grad(grad, ids, vocab, 0.7, 0, NAMES[tdt]))
    # added to what is there; rows that no token names keep their bits
    before = rand(6, vocab, cols, NAMES[tdt])
    acc = Guarded(vocab, cols, NAMES[tdt], 8, 0)
    acc.t.copy_(before)
    C.fsdp_embedding_grad(grad, ids, acc.t, w, scale=0.7, accumulate=True)
    R.agree("grad", acc.check(), R.embedding_grad(grad, ids, vocab, 0.7, 0, NAMES[tdt], before))
    work.check()
    named = torch.zeros(vocab + 1, dtype=torch.bool, device="cuda")
    l = ids.long()
    named[torch.where((l >= 0) & (l < vocab), l, vocab)] = True
    assert torch.equal(acc.t[~named[:vocab]], before[~named[:vocab]])


@pytest.mark.parametrize("n, vocab, kind", [(20000, 17, "uniform"), (9000, 40000, "hot"), (40000, 1000, "one"), (8193, 2 ** 17 + 5, "uniform"),
                                            (100003, 131, "wild"), (20000, 70000, "sorted"), (9000, 2 ** 19 + 3, "uniform"),
                                            (4097, 250, "hot"), (512, 100000, "hot")])
def test_embedding_grad_of_many_tokens_is_exact_on_whole_numbers(n, vocab, kind):
    # sums of small whole numbers are exact in any order: what is checked is
    # that every token reaches its row once, across the sort's blocks and the
    # chunks of the sums
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    grad = torch.randint(-8, 9, (n, 72), generator=g, device="cuda").float()
    ids = ids_of(8, n, vocab, kind)
    out = Guarded(vocab, 72, F32)
    work = Workspace(C.fsdp_embedding_grad_workspace(n, vocab, 72))
    C.fsdp_embedding_grad(grad, ids, out.t, work.t)
    work.check()
    l = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    want = torch.zeros(vocab + 1, 72, dtype=torch.float64, device="cuda").index_add_(0, l, grad.double())[:vocab]
    assert torch.equal(out.check().double(), want)


@pytest.mark.parametrize("most, n", [(5000, 4096), (20000, 16384), (20000, 4096), (16385, 16384), (40000, 600)])
def test_embedding_grad_of_fewer_tokens_than_the_workspace_was_sized_for(most, n):
    vocab, cols = 300, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(15)
    grad = torch.randint(-8, 9, (n, cols), generator=g, device="cuda").float()
    ids = ids_of(16, n, vocab, "hot")
    out, work = Guarded(vocab, cols, F32), Workspace(C.fsdp_embedding_grad_workspace(most, vocab, cols))
    C.fsdp_embedding_grad(grad, ids, out.t, work.t)
    work.check()
    want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, ids, grad.double())
    assert torch.equal(out.check().double(), want)


def test_embedding_grad_gives_equal_bits_and_keeps_other_rows_apart():
    n, vocab, cols = 30000, 500, 520
    grad, ids = rand(9, n, cols, BF16), ids_of(10, n, vocab, "hot")
    w = torch.empty(C.fsdp_embedding_grad_workspace(n, vocab, cols), dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0, 0xFF):
        w.fill_(fill)
        outs.append(Guarded(vocab, cols, F32))
        C.fsdp_embedding_grad(grad, ids, outs[-1].t, w)
    assert torch.equal(outs[0].check(), outs[1].check())
    # a NaN in one token's gradient stays in its row and its column
    t = int((ids == 1).nonzero()[17])
    grad[t, 5] = float("nan")
    got = torch.empty(vocab, cols, device="cuda")
    C.fsdp_embedding_grad(grad, ids, got, w)
    assert torch.isnan(got).nonzero().tolist() == [[1, 5]]
    got[1, 5] = outs[0].t[1, 5]
    assert torch.equal(got, outs[0].t)


def test_embedding_gradient_against_differences():
    # f = sum(c * embedding(table)): its change along a direction is the gradient's product with it, exactly, f being linear
    table, ids, c = rand(11, 60, 48, F32), ids_of(12, 400, 60, "wild"), rand(13, 400, 48, F32)
    grad = torch.empty_like(table)
    w = torch.empty(C.fsdp_embedding_grad_workspace(400, 60, 48), dtype=torch.uint8, device="cuda")
    C.fsdp_embedding_grad(c, ids, grad, w, scale=1.5)
    step = rand(14, 60, 48, F32)
    y0, y1 = torch.empty_like(c), torch.empty_like(c)
    C.fsdp_embedding(table, ids, y0, scale=1.5)
    C.fsdp_embedding((table + step), ids, y1, scale=1.5)
    got = float((c.double() * (y1.double() - y0.double())).sum())
    want = float((grad.double() * ((table + step).double() - table.double())).sum())
    mag = float((c.double().abs() * (y1.double().abs() + y0.double().abs())).sum())
    assert abs(got - want) <= 400 * R.U32 * mag


# ----------------------------------------------------------------- dropout

SIZES = [(700, 512, 0, 0), (90, 520, 0, 0), (600, 97, 0, 0), (1, 1, 0, 0), (3, 8, 0, 0), (5, 7, 0, 0), (2, 256, 0, 0), (37, 1000, 0, 0), (4, 511, 1, 3), (9, 2056, 8, 0), (130, 33, 0, 1),
         (1, 70001, 0, 0)]


@pytest.mark.parametrize("dt", NAMES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows, cols, pad, offset", SIZES)
def test_dropout(dt, residual, rows, cols, pad, offset):
    x = rand(1, rows, cols, NAMES[dt], pad=pad, offset=offset)
    res = rand(2, rows, cols, NAMES[dt], pad=8 - pad, offset=0) if residual else None
    for p, seed, draw in [(0.1, 0x0123456789ABCDEF, 3), (0.5, 1, 2 ** 32 - 1)]:
        out = Guarded(rows, cols, NAMES[dt], pad, (offset + 2) % 8)
        C.fsdp_dropout(x, out.t, p, seed, draw, residual=res)
        v, err, _ = R.dropout(x, res, p, seed, draw)
        R.agree("out", out.check(), (v, err))


@pytest.mark.parametrize("dt", NAMES)
def test_dropout_of_everything_and_nothing(dt):
    x, res = rand(1, 6, 100, NAMES[dt]), rand(2, 6, 100, NAMES[dt])
    out = torch.empty_like(x)
    C.fsdp_dropout(x, out, 0.0, 5)
    assert torch.equal(out, x)
    C.fsdp_dropout(x, out, 1e-9, 5)  # below the mask's step: nothing is dropped
    assert torch.equal(out, x)
    x[0, 0], x[1, 1], x[2, 2] = float("nan"), float("inf"), -float("inf")
    C.fsdp_dropout(x, out, 1.0, 5)
    assert bool((out == 0).all())
    C.fsdp_dropout(x, out, 1.0, 5, residual=res)
    assert torch.equal(out, res)


def test_dropout_hides_what_it_drops():
    # NaN, infinities and the type's lowest value at every dropped place
    rows, cols, p = 16, 300, 0.5
    x = rand(1, rows, cols, BF16)
    gone = torch.from_numpy(R.mask(rows, cols, p, 9, 1) == 0).cuda()
    clean = torch.empty_like(x)
    C.fsdp_dropout(x, clean, p, 9, 1)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF16).min):
        out = torch.empty_like(x)
        C.fsdp_dropout(torch.where(gone, torch.full_like(x, bad), x), out, p, 9, 1)
        assert torch.equal(out, clean)


@pytest.mark.parametrize("dt", NAMES)
@pytest.mark.parametrize("rows, cols, pad", [(7, 64, 0), (5, 77, 0), (300, 513, 1)])
def test_dropout_in_place(dt, rows, cols, pad):
    x, res = rand(1, rows, cols, NAMES[dt], pad=pad), rand(2, rows, cols, NAMES[dt], pad=pad)
    want = torch.empty(rows, cols, dtype=NAMES[dt], device="cuda")
    C.fsdp_dropout(x, want, 0.3, 4, 1, residual=res)
    a, b = Guarded(rows, cols, NAMES[dt], pad, 1), Guarded(rows, cols, NAMES[dt], pad, 1)
    a.t.copy_(x), b.t.copy_(res)
    C.fsdp_dropout(a.t, a.t, 0.3, 4, 1, residual=res)
    C.fsdp_dropout(x, b.t, 0.3, 4, 1, residual=b.t)
    assert torch.equal(a.check(), want) and torch.equal(b.check(), want)


def test_dropout_backward_is_the_same_mask_and_broadcast_inputs():
    x = rand(1, 9, 200, F32)
    y, ones = torch.empty_like(x), torch.ones(1, 200, device="cuda").expand(9, 200)
    C.fsdp_dropout(x, y, 0.4, 77, 5)
    g = torch.empty_like(x)
    C.fsdp_dropout(ones, g, 0.4, 77, 5)  # the derivative of the sum, from a row stride of 0
    assert torch.equal(y, x * g)


def test_dropout_of_a_tensor_of_three_dimensions():
    x = rand(1, 24, 40, BF16)
    a, b = torch.empty_like(x), torch.empty(2, 12, 40, dtype=BF16, device="cuda")
    C.fsdp_dropout(x, a, 0.2, 3)
    C.fsdp_dropout(x.contiguous().view(2, 12, 40), b, 0.2, 3)
    assert torch.equal(a, b.view(24, 40))


# -------------------------------------------------------------- layer norm

NORM_SIZES = [(1, 1, 0, 0), (3, 2, 0, 0), (5, 8, 0, 0), (9, 100, 0, 0), (33, 256, 8, 0), (4, 513, 0, 1), (7, 1024, 0, 0), (6, 1537, 1, 3),
              (3, 4096, 0, 0), (2, 5003, 0, 0), (3, 8192, 0, 0), (2, 16384, 0, 0), (2, 16391, 0, 0), (1, 40000, 0, 0), (700, 72, 0, 0)]
MODES = [(0.0, False), (0.0, True), (0.1, False), (0.25, True)]


# more rows than the GPU holds at once, for every number of granules a thread
MANY_ROWS = [(6000, 40, 0, 0), (5003, 201, 0, 1), (2000, 520, 0, 0), (400, 1000, 0, 0), (400, 1001, 0, 0), (380, 2500, 0, 0), (401, 4096, 8, 0),
             (310, 5003, 0, 0), (320, 8192, 0, 0), (310, 9000, 0, 0)]


@pytest.mark.parametrize("rows, cols, pad, offset", MANY_ROWS)
@pytest.mark.parametrize("dt", NAMES)
def test_layer_norm_of_many_rows(dt, rows, cols, pad, offset):
    x, res = rand(1, rows, cols, NAMES[dt], pad=pad, offset=offset), rand(2, rows, cols, NAMES[dt], pad=pad)
    w, b = vec(3, cols, NAMES[dt], 1.0), vec(4, cols, NAMES[dt])
    out, hid = Guarded(rows, cols, NAMES[dt], pad, offset), Guarded(rows, cols, NAMES[dt], pad, 0)
    mean, rstd = Guarded(1, rows, F32), Guarded(1, rows, F32)
    C.fsdp_layer_norm(x, w, b, out.t, mean.t, rstd.t, residual=res, hidden=hid.t, p=0.1, seed=21, draw=1)
    want = R.layer_norm(x, w, b, 1e-5, res, 0.1, 21, 1)
    for name, got in (("out", out), ("hidden", hid), ("mean", mean), ("rstd", rstd)):
        R.agree(name, got.check(), want[name])
    gx, gr = Guarded(rows, cols, NAMES[dt], pad, offset), Guarded(rows, cols, NAMES[dt], pad, 0)
    gw, gb = Guarded(1, cols, F32), Guarded(1, cols, F32)
    work = Workspace(C.fsdp_layer_norm_grad_workspace(rows, cols))
    C.fsdp_layer_norm_grad(x, hid.t, mean.t.view(-1), rstd.t.view(-1), w, gx.t, gw.t.view(-1), gb.t.view(-1), work.t, grad_hidden=res,
                           grad_residual=gr.t, p=0.1, seed=21, draw=1)
    work.check()
    want = R.layer_norm_grad(x, hid.t, mean.t.view(-1), rstd.t.view(-1), w, F32, res, 0.1, 21, 1)
    for name, got in (("grad_x", gx), ("grad_residual", gr), ("grad_weight", gw), ("grad_bias", gb)):
        R.agree(name, got.check(), want[name])


@pytest.mark.parametrize("dt, pdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows, cols, pad, offset", NORM_SIZES)
def test_layer_norm(dt, pdt, rows, cols, pad, offset):
    x = rand(1, rows, cols, NAMES[dt], pad=pad, offset=offset, shift=3.0)
    w, b = vec(3, cols, NAMES[pdt], 1.0), vec(4, cols, NAMES[pdt])
    for p, residual in MODES:
        res = rand(2, rows, cols, NAMES[dt], pad=pad) if residual else None
        out, hid = Guarded(rows, cols, NAMES[dt], pad, offset), Guarded(rows, cols, NAMES[dt], 3, 2)
        mean, rstd = Guarded(1, rows, F32), Guarded(1, rows, F32)
        C.fsdp_layer_norm(x, w, b, out.t, mean.t, rstd.t, residual=res, hidden=hid.t, p=p, seed=11, draw=2)
        want = R.layer_norm(x, w, b, 1e-5, res, p, 11, 2)
        for name, got in (("out", out), ("hidden", hid), ("mean", mean), ("rstd", rstd)):
            R.agree(name, got.check(), want[name])


def test_layer_norm_with_parts_left_out():
    x = rand(1, 5, 300, BF16)
    out = Guarded(5, 300, BF16)
    w, b = vec(3, 300, BF16, 1.0), vec(4, 300, BF16)
    for weight, bias in ((None, None), (w, None), (None, b)):
        C.fsdp_layer_norm(x, weight, bias, out.t, None, None, eps=0.0)
        R.agree("out", out.check(), R.layer_norm(x, weight, bias, 0.0)["out"])


def test_layer_norm_of_constant_and_loud_rows():
    # equal values: variance 0, out = bias; a large mean costs the variance nothing; other rows do not see a NaN
    x = rand(1, 6, 1000, F32)
    x[1] = 7.25
    x[2] += 10000.0
    x[3, 5] = float("nan")
    x[4, 999] = float("inf")
    w, b = vec(3, 1000, F32, 1.0), vec(4, 1000, F32)
    out, mean, rstd = Guarded(6, 1000, F32), Guarded(1, 6, F32), Guarded(1, 6, F32)
    C.fsdp_layer_norm(x, w, b, out.t, mean.t, rstd.t)
    got = out.check()
    assert torch.equal(got[1], b)
    assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[4]).all())
    keep = [0, 1, 2, 5]
    want = R.layer_norm(x[keep], w, b, 1e-5)
    R.agree("out", got[keep], want["out"])
    R.agree("mean", mean.t[0, keep], want["mean"])
    R.agree("rstd", rstd.t[0, keep], want["rstd"])


@pytest.mark.parametrize("cols", [1000, 1001, 8192, 20000])
def test_layer_norm_of_constant_rows_of_many_bits(cols):
    # sums of equal values that are not exact: mean and output within binary32's bounds, not equal to the value and the bias
    values = torch.tensor([0.64042264, -0.5356694, 0.1, 1.0 / 3.0, -7.0, 0.0], device="cuda")
    x = values[:, None].expand(-1, cols).contiguous()
    w, b = vec(3, cols, F32, 1.0), vec(4, cols, F32)
    out, mean, rstd = Guarded(len(values), cols, F32), Guarded(1, len(values), F32), Guarded(1, len(values), F32)
    C.fsdp_layer_norm(x, w, b, out.t, mean.t, rstd.t)
    want = R.layer_norm(x, w, b, 1e-5)
    for name, got in (("out", out), ("mean", mean), ("rstd", rstd)):
        R.agree(name, got.check(), want[name])
    assert torch.equal(out.t[4:], b.expand(2, cols)) and torch.equal(mean.t[0, 4:], values[4:])  # exact sums


@pytest.mark.parametrize("dt, pdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows, cols, pad, offset", NORM_SIZES)
def test_layer_norm_grad(dt, pdt, rows, cols, pad, offset):
    hid = rand(1, rows, cols, NAMES[dt], pad=pad, offset=offset, shift=2.0)
    g = rand(2, rows, cols, NAMES[dt], pad=3)
    mean = hid.float().mean(1)
    rstd = (hid.float().var(1, unbiased=False) + 1e-5).rsqrt()
    w = vec(3, cols, NAMES[pdt], 1.0)
    work = Workspace(C.fsdp_layer_norm_grad_workspace(rows, cols))
    for i, (p, residual) in enumerate(MODES):
        gh = rand(5, rows, cols, NAMES[dt], pad=pad) if residual else None
        gx, gr = Guarded(rows, cols, NAMES[dt], pad, offset), Guarded(rows, cols, NAMES[dt], 8, 0)
        gw, gb = Guarded(1, cols, NAMES[pdt], 0, 1), Guarded(1, cols, NAMES[pdt])
        before = (vec(6, cols, NAMES[pdt]), vec(7, cols, NAMES[pdt])) if i % 2 else (None, None)
        if i % 2:
            gw.t[0].copy_(before[0]), gb.t[0].copy_(before[1])
        C.fsdp_layer_norm_grad(g, hid, mean, rstd, w, gx.t, gw.t.view(-1), gb.t.view(-1), work.t, grad_hidden=gh, grad_residual=gr.t,
                               p=p, seed=11, draw=2, accumulate=bool(i % 2))
        work.check()
        want = R.layer_norm_grad(g, hid, mean, rstd, w, NAMES[pdt], gh, p, 11, 2, *before)
        for name, got in (("grad_x", gx), ("grad_residual", gr), ("grad_weight", gw), ("grad_bias", gb)):
            R.agree(name, got.check(), want[name])


def test_layer_norm_grad_of_many_rows_parts_left_out_and_no_rows():
    rows, cols = 5001, 96
    hid, g = rand(1, rows, cols, F32), rand(2, rows, cols, F32)
    mean = hid.mean(1)
    rstd = (hid.var(1, unbiased=False) + 1e-5).rsqrt()
    work = torch.empty(C.fsdp_layer_norm_grad_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    want = R.layer_norm_grad(g, hid, mean, rstd, None, F32)
    for left in ("none", "weight", "bias", "both"):
        gx, gw, gb = Guarded(rows, cols, F32), Guarded(1, cols, F32), Guarded(1, cols, F32)
        C.fsdp_layer_norm_grad(g, hid, mean, rstd, None, gx.t, None if left in ("weight", "both") else gw.t.view(-1),
                               None if left in ("bias", "both") else gb.t.view(-1), work)
        R.agree("grad_x", gx.check(), want["grad_x"])
        for name, t, gone in (("grad_weight", gw, ("weight", "both")), ("grad_bias", gb, ("bias", "both"))):
            t.check()
            if left in gone:
                assert bool((t.buf.view(torch.uint8) == 0x5A).all())
            else:
                R.agree(name, t.t, want[name])
    none = g[:0]
    gw, gb = Guarded(1, cols, F32), Guarded(1, cols, F32)
    C.fsdp_layer_norm_grad(none, none, mean[:0], rstd[:0], None, none.clone(), gw.t.view(-1), gb.t.view(-1), work[:0])
    assert bool((gw.check() == 0).all()) and bool((gb.check() == 0).all())


def test_layer_norm_gradient_against_differences():
    # f = sum(c * norm(residual + drop(x))) in 64 bits along a direction, by central differences
    rows, cols, p = 4, 60, 0.25
    x, res, c = rand(1, rows, cols, F32), rand(2, rows, cols, F32), rand(3, rows, cols, F32)
    w, b = vec(4, cols, F32, 1.0), vec(5, cols, F32)
    hid, out, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    C.fsdp_layer_norm(x, w, b, out, mean, rstd, residual=res, hidden=hid, p=p, seed=3, draw=4)
    gx, gr, gw, gb = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    work = torch.empty(C.fsdp_layer_norm_grad_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    C.fsdp_layer_norm_grad(c, hid, mean, rstd, w, gx, gw, gb, work, grad_residual=gr, p=p, seed=3, draw=4)
    rng = np.random.default_rng(0)
    k, cd = R.mask(rows, cols, p, 3, 4), R.f64(c)

    def f(x_, r_, w_, b_):
        h = r_ + k * x_
        d = h - h.mean(1, keepdims=True)
        return float((cd * (d / np.sqrt((d * d).mean(1, keepdims=True) + 1e-5) * w_ + b_)).sum())

    at = [R.f64(v) for v in (x, res, w, b)]
    for i, got in enumerate((gx, gr, gw, gb)):
        step = rng.standard_normal(at[i].shape)
        e = 1e-4
        up, down = [v + e * step * (j == i) for j, v in enumerate(at)], [v - e * step * (j == i) for j, v in enumerate(at)]
        want, have = (f(*up) - f(*down)) / (2 * e), float((R.f64(got) * step).sum())
        # third derivatives over e^2 and binary32 noise: both far below 1e-4 of the terms' size
        assert abs(want - have) <= 1e-4 * float(np.abs(R.f64(got) * step).sum())


# ------------------------------------------------------------ calls in use

def test_strides_past_32_bits():
    # two rows 2^31 elements and more apart in one buffer
    stride = 2 ** 31 + 8
    buf = torch.empty(2 * stride, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (2, 264), (stride, 1))
    x.copy_(rand(1, 2, 264, BF16))
    out = torch.as_strided(buf, (2, 264), (stride, 1), 1024)
    C.fsdp_dropout(x, out, 0.5, 1)
    v, err, _ = R.dropout(x, None, 0.5, 1, 0)
    R.agree("out", out, (v, err))
    mean, rstd = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    C.fsdp_layer_norm(x, None, None, out, mean, rstd)
    R.agree("out", out, R.layer_norm(x, None, None, 1e-5)["out"])
    ids = torch.tensor([1, 0, 1], device="cuda")
    y = Guarded(3, 264, BF16)
    C.fsdp_embedding(x, ids, y.t)
    assert torch.equal(y.check(), x[ids])
    w = torch.empty(C.fsdp_embedding_grad_workspace(3, 2, 264), dtype=torch.uint8, device="cuda")
    C.fsdp_embedding_grad(y.t, ids, out, w)
    R.agree("grad", out, R.embedding_grad(y.t, ids, 2, 1.0, 0, BF16))


@pytest.mark.parametrize("n", [500, 3000, 9000])  # the gradient in one kernel, and by a sort of one and of several blocks
def test_side_stream_and_graph(n):
    vocab, cols = 80, 136
    table, ids = rand(1, vocab, cols, BF16), ids_of(2, n, vocab, "uniform")
    w, b = vec(3, cols, BF16, 1.0), vec(4, cols, BF16)
    new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    emb, hid, out, gx, gt, gw, gb = new(n, cols), new(n, cols), new(n, cols), new(n, cols), new(vocab, cols), new(cols), new(cols)
    mean, rstd = new(n, dtype=F32), new(n, dtype=F32)
    wk1 = new(C.fsdp_embedding_grad_workspace(n, vocab, cols), dtype=torch.uint8)
    wk2 = new(C.fsdp_layer_norm_grad_workspace(n, cols), dtype=torch.uint8)

    def step(stream=None):
        C.fsdp_embedding(table, ids, emb, scale=2.0, stream=stream)
        C.fsdp_layer_norm(emb, w, b, out, mean, rstd, hidden=hid, p=0.1, seed=8, stream=stream)
        C.fsdp_layer_norm_grad(out, hid, mean, rstd, w, gx, gw, gb, wk2, p=0.1, seed=8, stream=stream)
        C.fsdp_embedding_grad(gx, ids, gt, wk1, scale=2.0, stream=stream)

    results = (emb, hid, out, mean, rstd, gx, gt, gw, gb)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in results:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b_) for a, b_ in zip(results, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in results:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b_) for a, b_ in zip(results, want))


def test_binding_refuses():
    x, ids = rand(1, 4, 16, BF16), torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.empty(4, 16, device="cuda")
    work = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    v, m = torch.empty(16, dtype=BF16, device="cuda"), torch.empty(4, device="cuda")
    for call in [
            lambda: C.fsdp_dropout(x, f, 0.1, 1), lambda: C.fsdp_dropout(x, x[:3], 0.1, 1), lambda: C.fsdp_dropout(x.t(), x.t(), 0.1, 1),
            lambda: C.fsdp_dropout(x.half(), x.half(), 0.1, 1), lambda: C.fsdp_dropout(x, x, 1.1, 1),
            lambda: C.fsdp_embedding(x, ids.float(), x), lambda: C.fsdp_embedding(x, ids[::2], x), lambda: C.fsdp_embedding(x, ids[:3], x),
            lambda: C.fsdp_embedding(x, ids.cpu(), x), lambda: C.fsdp_embedding_grad(x, ids, x, work[:100]),
            lambda: C.fsdp_embedding_grad(x, ids, f[:, :8], work),
            lambda: C.fsdp_layer_norm(x, v[:8], None, f.bfloat16(), None, None), lambda: C.fsdp_layer_norm(x, v, v.float(), f.bfloat16(), None, None),
            lambda: C.fsdp_layer_norm(x, v, v, f.bfloat16(), m.bfloat16(), None), lambda: C.fsdp_layer_norm(x, v, v, x, m, m),
            lambda: C.fsdp_layer_norm_grad(x, x.clone(), m, m, v, x.clone(), v, v, work[:64]),
            lambda: C.fsdp_layer_norm_grad(x, x.clone(), m[:3], m, v, x.clone(), v, v, work)]:
        before = C.fsdp_launch_count()
        with pytest.raises(C.FsdpError) as e:
            call()
        assert e.value.code == C.FSDP_ERR_INVALID_ARG and C.fsdp_launch_count() == before
