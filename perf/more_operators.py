"""The matrix operators of a feed-forward block's training, as cases to time and compare.

Three operators on the matrices that an HSDP unit shards: the gated
feed-forward block, whose full parameters an unshard gathers; its gradient,
which a gradient sync reduces; and the orthogonalisation of a matrix's update
by Newton-Schulz products, which an optimizer step applies to the shards.
``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package's calls.

    gate = x w_gate^T,  up = x w_up^T,  out = (act(gate) * up) w_down^T
    X_0 = G / (|G|_F + eps),  A = X X^T,  X <- a X + (b A + c A A) X,  out = scale X
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through the (2,4) layer's block: reading the weights is all there is
        {"name": "ffn_token", "op": "ffn", "tokens": 1, "hidden": 4096, "inner": 11008, "act": "silu", "train": False, "pad": 0},
        # a few tokens through the large layer's block
        {"name": "ffn_few", "op": "ffn", "tokens": 48, "hidden": 8192, "inner": 28672, "act": "silu", "train": False, "pad": 0},
        # odd sizes throughout, rows off the 16-byte grid, projections kept for the gradient
        {"name": "ffn_odd", "op": "ffn", "tokens": 1001, "hidden": 1111, "inner": 3001, "act": "gelu", "train": True, "pad": 3},
        # a training batch through the (2,4) layer's block
        {"name": "ffn_train", "op": "ffn", "tokens": 16384, "hidden": 4096, "inner": 11008, "act": "silu", "train": True, "pad": 0},
        # a full batch through the large layer's block
        {"name": "ffn_large", "op": "ffn", "tokens": 16384, "hidden": 8192, "inner": 28672, "act": "silu", "train": False, "pad": 0},
        # the gradient of a short sequence: writing the weights' gradients is most of it
        {"name": "ffn_grad_few", "op": "ffn_grad", "tokens": 64, "hidden": 4096, "inner": 11008, "act": "silu", "pad": 0},
        # the gradient at odd sizes
        {"name": "ffn_grad_odd", "op": "ffn_grad", "tokens": 517, "hidden": 777, "inner": 2049, "act": "gelu", "pad": 5},
        # a batch's gradient at the large layer's sizes
        {"name": "ffn_grad_large", "op": "ffn_grad", "tokens": 8192, "hidden": 8192, "inner": 28672, "act": "silu", "pad": 0},
        # a small matrix's update: a chain of products, each of which is over at once
        {"name": "ortho_few", "op": "ortho", "rows": 128, "cols": 384, "dtype": "bf16", "kind": "noise", "pad": 0},
        # a tall matrix of odd sizes in fp32
        {"name": "ortho_odd", "op": "ortho", "rows": 2049, "cols": 1111, "dtype": "f32", "kind": "spikes", "pad": 1},
        # the (2,4) layer's down projection, its momentum kept in fp32
        {"name": "ortho_layer", "op": "ortho", "rows": 4096, "cols": 11008, "dtype": "f32", "kind": "spikes", "pad": 0},
        # the large layer's gate projection
        {"name": "ortho_large", "op": "ortho", "rows": 28672, "cols": 8192, "dtype": "bf16", "kind": "spikes", "pad": 0},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, high):
    """Half of them multiples of 64, as widths of layers are, the others any length from one up."""
    return 64 * _log(rng, 1, high // 64) if rng.random() < 0.5 else _log(rng, 1, high)


def draw(rng):
    op, pad = rng.choice(["ffn", "ffn_grad", "ortho"]), rng.choice([0, 0, 0, 8, 3])
    if op == "ortho":
        rows, cols = _width(rng, 8192), _width(rng, 28672)
        if rng.random() < 0.5:
            rows, cols = cols, rows
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"]),
                "kind": rng.choice(["noise", "spikes", "spikes"]), "pad": pad}
    c = {"op": op, "tokens": _log(rng, 1, 16384 if op == "ffn" else 8192), "hidden": _width(rng, 8192), "inner": _width(rng, 28672),
         "act": rng.choice(["silu", "silu", "gelu", "relu"]), "pad": pad}
    if op == "ffn":
        c["train"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- inputs

def _values(gen, rows, cols, pad, std=1.0):
    """Activations: normal values, a mean that is not zero and a few loud columns; `pad` widens the row stride."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda").mul_(std)
    loud = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device="cuda")
    x[:, loud] *= 4.0
    return (x + 0.1 * std).to(torch.bfloat16)[:, :cols]


def _weight(gen, rows, cols):
    return (torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, pad = {"case": case}, case["pad"]
    if case["op"] == "ortho":
        m, n = case["rows"], case["cols"]
        g = torch.randn(m, n + pad, generator=gen, device="cuda")
        if case["kind"] == "spikes":  # a batch's gradient: a few strong directions over noise
            k = min(m, n, 8)
            left = torch.randn(m, k, generator=gen, device="cuda") * torch.logspace(0, -1, k, device="cuda")
            g = g.mul_(0.1).add_(left @ torch.randn(k, n + pad, generator=gen, device="cuda"))
        s["x"] = (g * 1e-3).to(DTYPES[case["dtype"]])[:, :n]
        s["scale"] = math.sqrt(max(1.0, m / n))
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        return s
    t, d, f = case["tokens"], case["hidden"], case["inner"]
    s["x"] = _values(gen, t, d, pad)
    s["w_gate"], s["w_up"], s["w_down"] = _weight(gen, f, d), _weight(gen, f, d), _weight(gen, d, f)
    if case["op"] == "ffn":
        s["out"] = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
        s["gate"], s["up"] = (torch.empty(t, f, dtype=torch.bfloat16, device="cuda") if case["train"] else None for _ in range(2))
        return s
    # what the forward pass kept
    s["gate"], s["up"] = s["x"] @ s["w_gate"].t(), s["x"] @ s["w_up"].t()
    s["grad_out"] = _values(gen, t, d, pad, 1e-2)
    s["grad_x"] = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    for name in ("w_gate", "w_up", "w_down"):
        s["grad_" + name] = torch.empty_like(s[name])
    return s


# ------------------------------------------------------------- plain forms

def _act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.where(z <= 0, torch.zeros_like(z), z)


def _slope(name, z):
    """The activation's derivative."""
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))


def _plain(s):
    c = s["case"]
    if c["op"] == "ortho":
        a, b, k = COEFFICIENTS
        x = s["x"].float()
        x = x / (x.norm() + EPS)
        tall = c["rows"] > c["cols"]
        x = x.t() if tall else x
        for _ in range(STEPS):
            g = x @ x.t()
            x = a * x + (b * g + k * (g @ g)) @ x
        return ((x.t() if tall else x) * s["scale"]).to(torch.bfloat16)
    x, w_gate, w_up, w_down = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    if c["op"] == "ffn":
        gate, up = x @ w_gate.t(), x @ w_up.t()
        y = ((_act(c["act"], gate) * up) @ w_down.t()).to(torch.bfloat16)
        return {"y": y, "gate": gate.to(torch.bfloat16), "up": up.to(torch.bfloat16)} if c["train"] else {"y": y}
    gate, up, grad = s["gate"].float(), s["up"].float(), s["grad_out"].float()
    h = grad @ w_down
    act = _act(c["act"], gate)
    g_gate, g_up = h * up * _slope(c["act"], gate), h * act
    out = {"x": g_gate @ w_gate + g_up @ w_up, "w_gate": g_gate.t() @ x, "w_up": g_up.t() @ x, "w_down": grad.t() @ (act * up)}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


# ------------------------------------------------------- the package's calls

def _own(s):
    from hsdp_sharded_parameter_gb300 import capi as C

    c = s["case"]
    if c["op"] == "ortho":
        if "work" not in s:  # the scratch memory that a training loop keeps
            s["work"] = torch.empty(C.fsdp_orthogonalize_workspace(c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
        C.fsdp_orthogonalize(s["x"], s["out"], s["work"], steps=STEPS, coefficients=COEFFICIENTS, scale=s["scale"], eps=EPS)
        return s["out"]
    aligned = all(n % 8 == 0 for n in (c["hidden"], c["inner"], c["pad"]))
    if c["op"] == "ffn":
        if "work" not in s:
            n = C.fsdp_gated_ffn_workspace(c["tokens"], c["hidden"], c["inner"], aligned=aligned)
            s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        C.fsdp_gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["out"], s["work"], activation=c["act"], gate=s["gate"],
                         up=s["up"])
        return {"y": s["out"], "gate": s["gate"], "up": s["up"]} if c["train"] else {"y": s["out"]}
    if "work" not in s:
        n = C.fsdp_gated_ffn_grad_workspace(c["tokens"], c["hidden"], c["inner"], aligned=aligned)
        s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    C.fsdp_gated_ffn_grad(s["grad_out"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"], s["grad_x"],
                          s["grad_w_gate"], s["grad_w_up"], s["grad_w_down"], s["work"], activation=c["act"])
    return {"x": s["grad_x"], "w_gate": s["grad_w_gate"], "w_up": s["grad_w_up"], "w_down": s["grad_w_down"]}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 8e12:  # over about 20 seconds at the rate of 64-bit products
        return None
    s = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, k = COEFFICIENTS
        x = s["x"].double()
        x = x / (x.square().sum().sqrt() + EPS)
        wide = case["rows"] <= case["cols"]
        for _ in range(STEPS):  # the smaller side's products, from the left or from the right
            g = x @ x.mT if wide else x.mT @ x
            p = b * g + k * g @ g
            p.diagonal().add_(a)
            x = p @ x if wide else x @ p
        return x * s["scale"]
    t, act = case["tokens"], case["act"]
    w = {k: s[k].double() for k in ("w_gate", "w_up", "w_down")}
    x = s["x"].double()
    if case["op"] == "ffn":
        gate, up = x @ w["w_gate"].mT, x @ w["w_up"].mT
    else:
        gate, up = s["gate"].double(), s["up"].double()
    if act == "silu":
        e = torch.exp(-gate.abs())
        p = torch.where(gate >= 0, 1 / (1 + e), e / (1 + e))
        slope = p + gate * e / (1 + e) ** 2
    elif act == "gelu":
        p = 0.5 * torch.special.erfc(-gate / math.sqrt(2.0))
        slope = p + gate * torch.exp(-gate * gate / 2) / math.sqrt(2 * math.pi)
    else:
        p = (gate > 0).double()
        slope = p
    value = gate * p
    if case["op"] == "ffn":
        y = torch.empty(t, case["hidden"], dtype=torch.float64, device="cuda")
        for first in range(0, t, 2048):
            y[first : first + 2048] = (value[first : first + 2048] * up[first : first + 2048]) @ w["w_down"].mT
        return {"y": y, "gate": gate, "up": up} if case["train"] else {"y": y}
    grad = s["grad_out"].double()
    through = grad @ w["w_down"]
    down = grad.mT @ (value * up)
    d_up = through * value
    d_gate = through.mul_(up).mul_(slope)
    return {"x": d_gate @ w["w_gate"] + d_up @ w["w_up"], "w_gate": d_gate.mT @ x, "w_up": d_up.mT @ x, "w_down": down}


# ------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; the products' operations, half of them where the result is symmetric."""
    if case["op"] == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        # X X^T and A A are symmetric, (b A + c A A) X is not
        return {"bytes": m * n * (BYTES[case["dtype"]] + 2), "flops": STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)}
    t, d, f = case["tokens"], case["hidden"], case["inner"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (2 * t * d + 3 * d * f + (2 * t * f if case["train"] else 0)), "flops": 6 * t * d * f}
    # grad_out, x, gate, up and the weights in, the gradients of x and of the weights out
    return {"bytes": 2 * (3 * t * d + 2 * t * f + 6 * d * f), "flops": 12 * t * d * f}
