"""The training operators beside the sharded data path, as cases to time and compare.

Three operators, forward and backward, the ones whose full parameters an HSDP
unit gathers and whose full gradients it reduces: the embedding lookup with a
scale and its gradient by sorted tokens, dropout from a counter-based
generator, and layer norm with the dropout and residual addition ahead of it.
``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package's calls.

The mask of a dropout is a function of (seed, draw, row, column) alone: the
eight 16-bit halves of one Philox4x32-10 block with the counter
(column // 8, row low, row high, draw) and the key (seed low, seed high) decide
on eight neighbouring columns, low half first; an element is kept where its
half is below K = round((1 - p) * 65536), and then scaled by 65536 / K.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the last few tokens of a short batch: one launch's latency
        {"name": "embedding_few", "op": "embedding", "tokens": 8, "vocab": 32000, "cols": 4096, "dtype": "bf16",
         "out": "bf16", "ids": "uniform", "index": "i64", "pad": 0},
        # a full batch over a large vocabulary at the hidden size of the large layer
        {"name": "embedding_batch", "op": "embedding", "tokens": 32768, "vocab": 131072, "cols": 8192, "dtype": "bf16",
         "out": "bf16", "ids": "zipf", "index": "i64", "pad": 0},
        # a table kept in fp32 and looked up for bf16 compute, odd sizes throughout
        {"name": "embedding_odd", "op": "embedding", "tokens": 5003, "vocab": 50021, "cols": 1111, "dtype": "f32",
         "out": "bf16", "ids": "zipf", "index": "i32", "pad": 0},
        # the gradient of a small odd table, most tokens in a few rows
        {"name": "embedding_grad_few", "op": "embedding_grad", "tokens": 300, "vocab": 4099, "cols": 1027, "dtype": "f32",
         "out": "f32", "ids": "hot", "index": "i32", "pad": 0},
        # the gradient of a batch at the hidden size of the (2,4) layer
        {"name": "embedding_grad_batch", "op": "embedding_grad", "tokens": 16384, "vocab": 32000, "cols": 4096,
         "dtype": "bf16", "out": "bf16", "ids": "zipf", "index": "i64", "pad": 0},
        # the largest: a large vocabulary's gradient in fp32 from bf16 activations
        {"name": "embedding_grad_large", "op": "embedding_grad", "tokens": 65536, "vocab": 131072, "cols": 8192,
         "dtype": "bf16", "out": "f32", "ids": "zipf", "index": "i64", "pad": 0},
        # a small activation in fp32
        {"name": "dropout_few", "op": "dropout", "rows": 37, "cols": 1000, "dtype": "f32", "p": 0.25, "residual": False, "pad": 0},
        # a sublayer's output dropped and added to the residual stream
        {"name": "dropout_add_large", "op": "dropout", "rows": 32768, "cols": 8192, "dtype": "bf16", "p": 0.1, "residual": True, "pad": 0},
        # a few rows: latency of one launch
        {"name": "norm_few", "op": "norm", "rows": 16, "cols": 4096, "dtype": "bf16", "param": "bf16", "p": 0.0,
         "residual": False, "pad": 0},
        # a block of the large layer: dropout, residual and norm in one pass
        {"name": "norm_block", "op": "norm", "rows": 16384, "cols": 8192, "dtype": "bf16", "param": "bf16", "p": 0.1,
         "residual": True, "pad": 0},
        # odd sizes in fp32, the plain norm's gradient
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 3001, "cols": 1537, "dtype": "f32", "param": "f32", "p": 0.0,
         "residual": False, "pad": 0},
        # the gradient of that block: norm, residual stream, dropout, weight and bias
        {"name": "norm_grad_block", "op": "norm_grad", "rows": 16384, "cols": 8192, "dtype": "bf16", "param": "bf16", "p": 0.1,
         "residual": True, "pad": 0},
    ]


def _log(rng, low, high):
    n = min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))
    return n + (n in (48, 3072))  # neither is a size of these cases


def _cols(rng):
    """Half of them multiples of 64, as hidden sizes are, the others any length from one up."""
    if rng.random() < 0.5:
        return 64 * _log(rng, 1, 128)
    return _log(rng, 1, 8192)


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "embedding_grad", "dropout", "norm", "norm_grad"])
    cols, dtype = _cols(rng), rng.choice(["bf16", "bf16", "f32"])
    pad = rng.choice([0, 0, 0, 8, 3])
    if op.startswith("embedding"):
        out = rng.choice([dtype, dtype, "f32" if op == "embedding_grad" else "bf16"])
        return {"op": op, "tokens": _log(rng, 1, 65536 if op == "embedding_grad" else 32768), "vocab": _log(rng, 2, 131072),
                "cols": cols, "dtype": dtype, "out": out, "ids": rng.choice(["zipf", "zipf", "uniform", "hot"]),
                "index": rng.choice(["i64", "i64", "i32"]), "pad": pad}
    rows = _log(rng, 1, 32768 if op == "dropout" else 16384)
    c = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "p": rng.choice([0.0, 0.1, 0.1, 0.25, 0.5]),
         "residual": rng.random() < 0.5, "pad": pad}
    if op == "dropout":
        c["p"] = c["p"] or 0.1
        return c
    c["param"] = rng.choice([dtype, "f32"])
    return c


# ----------------------------------------------------------------- inputs

def _values(gen, rows, cols, dtype, pad, std=1.0):
    """Activations: normal values, a mean that is not zero and a few loud columns; `pad` widens the row stride."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda").mul_(std)
    loud = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device="cuda")
    x[:, loud] *= 4.0
    return (x + 0.1 * std).to(DTYPES[dtype])[:, :cols]


def _ids(gen, case):
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["ids"] == "uniform":
        ids = (u * vocab).long()
    else:
        # ranks fall as 1/rank, as words do; "hot": nine in ten of them among the first three ranks
        rank = torch.exp(u * math.log(vocab + 1.0)).long() - 1
        if case["ids"] == "hot":
            few = torch.rand(n, generator=gen, device="cuda") < 0.9
            rank = torch.where(few, rank % 3, rank)
        ids = (rank.clamp(0, vocab - 1) * 7919) % vocab  # spread over the table
    # one token in 32 is padding: it names no row
    ids = torch.where(torch.rand(n, generator=gen, device="cuda") < 1 / 32, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["index"] == "i32" else torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype, pad, cols = case["op"], case["dtype"], case["pad"], case["cols"]
    s = {"case": case}
    if op.startswith("embedding"):
        s["ids"] = _ids(gen, case)
        s["scale"] = math.sqrt(cols)
        if op == "embedding":
            s["table"] = _values(gen, case["vocab"], cols, dtype, 0, 0.02)
            s["out"] = torch.empty(case["tokens"], cols, dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["grad_out"] = _values(gen, case["tokens"], cols, dtype, pad, 1e-2)
            s["grad_table"] = torch.empty(case["vocab"], cols, dtype=DTYPES[case["out"]], device="cuda")
        return s
    rows = case["rows"]
    s.update(p=case["p"], seed=seed * 0x9E3779B1 % (1 << 40), draw=seed % 1000, eps=1e-5)
    like = lambda: torch.empty(rows, cols, dtype=DTYPES[dtype], device="cuda")  # noqa: E731
    if op != "norm_grad":
        s["x"] = _values(gen, rows, cols, dtype, pad)
        s["residual"] = _values(gen, rows, cols, dtype, pad) if case["residual"] else None
        s["out"] = like()
    if op == "dropout":
        return s
    s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(DTYPES[case["param"]])
    s["bias"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(DTYPES[case["param"]])
    if op == "norm":
        s["hidden"] = like() if case["residual"] or case["p"] > 0 else None
        s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
        return s
    s["hidden"] = _values(gen, rows, cols, dtype, pad)
    s["mean"] = s["hidden"].float().mean(1)
    s["rstd"] = (s["hidden"].float() - s["mean"][:, None]).square().mean(1).add(s["eps"]).rsqrt()
    s["grad_out"] = _values(gen, rows, cols, dtype, pad, 1e-2)
    s["grad_hidden"] = _values(gen, rows, cols, dtype, pad, 1e-2) if case["residual"] else None
    s["grad_residual"] = like() if case["residual"] and case["p"] > 0 else None
    s["grad_x"] = like()
    s["grad_weight"], s["grad_bias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
    return s


# ------------------------------------------------------------- plain forms

def _keep(rows, cols, p, seed, draw):
    """(kept or not, the scale of what is kept), by 32 x 32 -> 64 bit products that wrap in int64."""
    limit = round((1.0 - p) * 65536)
    blocks = (cols + 7) // 8
    c0 = torch.arange(blocks, device="cuda")[None, :].expand(rows, blocks)
    r = torch.arange(rows, device="cuda")[:, None].expand(rows, blocks)
    c1, c2, c3 = r & M32, r >> 32, torch.full_like(c0, draw)
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & M32) ^ c1 ^ k0, b & M32, (a >> 32 & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    halves = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], dim=-1)
    return halves.reshape(rows, blocks * 8)[:, :cols] < limit, 65536.0 / max(limit, 1)


def _dropped(x, s):
    if s["p"] == 0:
        return x
    keep, scale = _keep(x.shape[0], x.shape[1], s["p"], s["seed"], s["draw"])
    return torch.where(keep, x * scale, torch.zeros_like(x))


def _plain(s):
    c = s["case"]
    if c["op"] == "embedding":
        named = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        rows = s["table"][s["ids"].long().clamp(0, c["vocab"] - 1)].float() * s["scale"]
        return torch.where(named[:, None], rows, torch.zeros_like(rows)).to(DTYPES[c["out"]])
    if c["op"] == "embedding_grad":
        named = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        total = torch.zeros(c["vocab"] + 1, c["cols"], device="cuda")
        total.index_add_(0, torch.where(named, s["ids"].long(), c["vocab"]), s["grad_out"].float() * s["scale"])
        return total[: c["vocab"]].to(DTYPES[c["out"]])
    dtype = DTYPES[c["dtype"]]
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), s)
        return (y if s["residual"] is None else y + s["residual"].float()).to(dtype)
    if c["op"] == "norm":
        h = _dropped(s["x"].float(), s)
        h = h if s["residual"] is None else h + s["residual"].float()
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + s["eps"])
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return {"y": y.to(dtype), "hidden": None if s["hidden"] is None else h.to(dtype), "mean": mean, "rstd": rstd}
    g = s["grad_out"].float()
    unit = (s["hidden"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    gw = g * s["weight"].float()
    total = s["rstd"][:, None] * (gw - gw.mean(1, keepdim=True) - unit * (gw * unit).mean(1, keepdim=True))
    if s["grad_hidden"] is not None:
        total = total + s["grad_hidden"].float()
    param = DTYPES[c["param"]]
    return {"x": _dropped(total, s).to(dtype), "residual": None if s["grad_residual"] is None else total.to(dtype),
            "weight": (g * unit).sum(0).to(param), "bias": g.sum(0).to(param)}


# ------------------------------------------------------- the package's calls

def _own(s):
    from hsdp_sharded_parameter_gb300 import capi as C

    c = s["case"]
    if c["op"] == "embedding":
        C.fsdp_embedding(s["table"], s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if c["op"] == "embedding_grad":
        if "work" not in s:  # the scratch memory that a training loop keeps
            n = C.fsdp_embedding_grad_workspace(c["tokens"], c["vocab"], c["cols"])
            s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        C.fsdp_embedding_grad(s["grad_out"], s["ids"], s["grad_table"], s["work"], scale=s["scale"])
        return s["grad_table"]
    if c["op"] == "dropout":
        C.fsdp_dropout(s["x"], s["out"], s["p"], s["seed"], s["draw"], residual=s["residual"])
        return s["out"]
    if c["op"] == "norm":
        C.fsdp_layer_norm(s["x"], s["weight"], s["bias"], s["out"], s["mean"], s["rstd"], eps=s["eps"],
                          residual=s["residual"], hidden=s["hidden"], p=s["p"], seed=s["seed"], draw=s["draw"])
        return {"y": s["out"], "hidden": s["hidden"], "mean": s["mean"], "rstd": s["rstd"]}
    if "work" not in s:
        s["work"] = torch.empty(C.fsdp_layer_norm_grad_workspace(c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
    C.fsdp_layer_norm_grad(s["grad_out"], s["hidden"], s["mean"], s["rstd"], s["weight"], s["grad_x"], s["grad_weight"],
                           s["grad_bias"], s["work"], grad_hidden=s["grad_hidden"], grad_residual=s["grad_residual"],
                           p=s["p"], seed=s["seed"], draw=s["draw"])
    return {"x": s["grad_x"], "residual": s["grad_residual"], "weight": s["grad_weight"], "bias": s["grad_bias"]}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------- in 64 bits

def _mul32(a, m):
    """(high, low) words of a 32 x 32 bit product, by 16-bit limbs."""
    al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = (al * ml >> 16) + (ah * ml & 0xFFFF) + (al * mh & 0xFFFF)
    low = (al * ml & 0xFFFF) | (mid & 0xFFFF) << 16
    return (ah * mh + (ah * ml >> 16) + (al * mh >> 16) + (mid >> 16)), low


def _factor(rows, cols, s):
    """What dropout multiplies each element by, in 64 bits."""
    limit, n = round((1.0 - s["p"]) * 65536), -(-cols // 8)
    out = torch.empty(rows, n, 8, dtype=torch.float64, device="cuda")
    for first in range(0, rows, 4096):
        m = min(4096, rows - first)
        row = torch.arange(first, first + m, device="cuda").repeat_interleave(n)
        c = [torch.arange(n, device="cuda").repeat(m), row % 2**32, row // 2**32, torch.zeros_like(row) + s["draw"]]
        key = [s["seed"] % 2**32, s["seed"] // 2**32]
        for _ in range(10):
            h0, l0 = _mul32(c[0], 0xD2511F53)
            h1, l1 = _mul32(c[2], 0xCD9E8D57)
            c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
        for j in range(8):
            half = c[j // 2] // (65536 if j % 2 else 1) % 65536
            out[first : first + m, :, j] = (half < limit).double().mul(65536 / max(limit, 1)).reshape(m, n)
    return out.reshape(rows, n * 8)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    ids, op = s.get("ids"), case["op"]
    if op == "embedding":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(ids >= 0).reshape(-1)
        out[at] = s["table"][ids[at].long()].double() * s["scale"]
        return out
    if op == "embedding_grad":
        out = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(ids >= 0).reshape(-1)
        return out.index_add_(0, ids[at].long(), s["grad_out"][at].double()).mul_(s["scale"])
    rows, cols = case["rows"], case["cols"]
    factor = _factor(rows, cols, s) if case["p"] > 0 else 1.0
    if op != "norm_grad":
        h = s["x"].double() * factor
        if s["residual"] is not None:
            h += s["residual"].double()
        if op == "dropout":
            return h
        mean, var = h.mean(1), h.var(1, unbiased=False)
        y = (h - mean[:, None]) / torch.sqrt(var + s["eps"])[:, None] * s["weight"].double() + s["bias"].double()
        return {"y": y, "hidden": None if s["hidden"] is None else h, "mean": mean, "rstd": 1 / torch.sqrt(var + s["eps"])}
    g, rstd = s["grad_out"].double(), s["rstd"].double()[:, None]
    unit = (s["hidden"].double() - s["mean"].double()[:, None]) * rstd
    gw = g * s["weight"].double()
    total = (gw * cols - gw.sum(1, keepdim=True) - unit * (gw * unit).sum(1, keepdim=True)) * rstd / cols
    if s["grad_hidden"] is not None:
        total += s["grad_hidden"].double()
    return {"x": total * factor, "residual": None if s["grad_residual"] is None else total,
            "weight": (g * unit).sum(0), "bias": g.sum(0)}


# ------------------------------------------------------------------- work

def _distinct(case):
    """How many rows of the table the ids name, on average."""
    n, vocab = case["tokens"] * 31 / 32, case["vocab"]
    if case["ids"] == "uniform":
        share = torch.full((vocab,), 1.0 / vocab, dtype=torch.float64)
    else:
        k = torch.arange(1, vocab + 1, dtype=torch.float64)
        share = torch.log1p(1 / k) / math.log(vocab + 1)
        if case["ids"] == "hot":
            few = torch.zeros(min(3, vocab), dtype=torch.float64).index_add_(0, (k.long() - 1) % min(3, vocab), share)
            share *= 0.1
            share[:3] += 0.9 * few
    return float((1 - (1 - share.clamp(max=1 - 1e-12)) ** n).sum())


def work(case):
    """Each input read once, each output written once; a dropped element's generator is counted at 10 operations."""
    op, cols, b = case["op"], case["cols"], BYTES[case["dtype"]]
    if op.startswith("embedding"):
        n, ids = case["tokens"], case["tokens"] * (4 if case["index"] == "i32" else 8)
        if op == "embedding":
            # the rows that are looked up, each once
            return {"bytes": ids + _distinct(case) * cols * b + n * cols * BYTES[case["out"]], "flops": n * cols}
        # the gradients of the tokens that name a row, and the whole table's
        return {"bytes": ids + n * 31 / 32 * cols * b + case["vocab"] * cols * BYTES[case["out"]], "flops": 2 * n * cols}
    n = case["rows"] * cols
    draws = 10 * n if case["p"] > 0 else 0
    if op == "dropout":
        return {"bytes": n * b * (3 if case["residual"] else 2), "flops": 2 * n + draws}
    params = 2 * cols * BYTES[case["param"]]
    if op == "norm":
        streams = 2 + (case["residual"] or 0) + (1 if case["residual"] or case["p"] > 0 else 0)
        return {"bytes": n * b * streams + params + 8 * case["rows"], "flops": 8 * n + draws}
    streams = 3 + (1 if case["residual"] else 0) + (1 if case["residual"] and case["p"] > 0 else 0)
    return {"bytes": n * b * streams + params + params // 2 + 8 * case["rows"], "flops": 14 * n + draws}
