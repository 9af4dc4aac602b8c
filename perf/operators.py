"""Cases of the language-model training operators: what they compute in plain
torch operations, the calls a user makes of the library, and the work each
cannot do without.

Four operators of one training step around the sparsifier:

* ``lookup``: rows of an embedding table, out[t] = scale * table[token[t]]; a
  negative token is a masked place and gives a row of zeros.
* ``grad``: the table's gradient, out[v] (+)= scale * sum of grad_out[t] over
  the places t with token[t] == v.
* ``orthogonalise``: the Newton-Schulz iteration X <- a X + (b A + c A^2) X
  with A = X X^T, from X = G / (|G|_F + eps).
* ``muon``: momentum m <- beta m + g, u = g + beta m, O = orthogonalise(u),
  w <- (1 - lr wd) w - lr s O with s = sqrt(max(1, rows / cols)).
"""
import math

import numpy as np
import torch

own = False

STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
LR, BETA, DECAY = 0.02, 0.95, 0.01
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "int32": torch.int32,
         "int64": torch.int64}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2, "int32": 4, "int64": 8}


def _lookup(T, V, D, table, out, ids="int64", scale=1.0, masked=0.0):
    return {"op": "lookup", "T": T, "V": V, "D": D, "table": table, "out": out, "ids": ids, "scale": scale,
            "masked": masked}


def _grad(T, V, D, grad, out, ids="int64", scale=1.0, masked=0.0, accumulate=False):
    return {"op": "grad", "T": T, "V": V, "D": D, "grad": grad, "out": out, "ids": ids, "scale": scale,
            "masked": masked, "accumulate": accumulate}


def _orthogonalise(batch, rows, cols, x, noise=0.3):
    return {"op": "orthogonalise", "batch": batch, "rows": rows, "cols": cols, "x": x, "noise": noise}


def _muon(batch, rows, cols, grad, weight, noise=0.3):
    return {"op": "muon", "batch": batch, "rows": rows, "cols": cols, "grad": grad, "weight": weight, "noise": noise}


def listed():
    return [
        # one generated token's row, scaled by sqrt(D): latency
        dict(_lookup(1, 32_000, 4_096, "bf16", "bf16", scale=64.0), name="lookup one token"),
        # a small batch from an fp32 table of odd width, some places masked
        dict(_lookup(4_099, 50_001, 1_001, "fp32", "fp32", "int32", scale=0.37, masked=0.05), name="lookup odd rows"),
        # a training batch of long sequences over a large vocabulary
        dict(_lookup(131_072, 128_000, 2_048, "bf16", "bf16"), name="lookup long batch"),
        # a toy model's whole embedding gradient: latency
        dict(_grad(512, 1_001, 130, "fp32", "fp32", "int32", scale=0.37, masked=0.05), name="grad small"),
        # the dense fp32 gradient that an error-feedback step over 25.6M entries takes
        dict(_grad(16_384, 25_000, 1_024, "bf16", "fp32"), name="grad 25.6M table"),
        # a micro-batch's gradient added to what earlier ones left, large vocabulary
        dict(_grad(131_072, 128_000, 2_048, "bf16", "fp32", masked=0.02, accumulate=True), name="grad accumulate long"),
        # one small projection: latency
        dict(_orthogonalise(1, 128, 128, "bf16"), name="orthogonalise small"),
        # odd sizes, fp32 in and out
        dict(_orthogonalise(1, 1_000, 1_533, "fp32"), name="orthogonalise odd fp32"),
        # a large square projection
        dict(_orthogonalise(1, 4_096, 4_096, "bf16"), name="orthogonalise 4096"),
        # a small model's layer with fp32 weights
        dict(_muon(1, 256, 768, "fp32", "fp32"), name="muon small fp32"),
        # the square projections of eight layers, stacked
        dict(_muon(8, 1_024, 1_024, "bf16", "bf16"), name="muon eight layers"),
        # a feed-forward layer's tall matrix
        dict(_muon(1, 8_192, 2_048, "bf16", "bf16"), name="muon tall"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lookup", "grad", "orthogonalise", "muon"))
    if op in ("lookup", "grad"):
        T, V, D = _between(rng, 1, 131_072), _between(rng, 2, 128_000), _between(rng, 1, 4_096)
        while T * D > 131_072 * 2_048 or V * D > 128_000 * 2_048:
            D = (D + 1) // 2
        types = ("fp32", "bf16", "fp16")
        ids, scale = rng.choice(("int32", "int64")), rng.choice((1.0, 0.37, math.sqrt(D)))
        masked = rng.choice((0.0, 0.05, 0.5))
        if op == "lookup":
            return _lookup(T, V, D, rng.choice(types), rng.choice(types), ids, scale, masked)
        return _grad(T, V, D, rng.choice(types), rng.choice(types), ids, scale, masked, rng.random() < 0.5)
    rows, cols, batch = _between(rng, 4, 8_192), _between(rng, 4, 8_192), _between(rng, 1, 32)
    while batch > 1 and batch * rows * cols * min(rows, cols) > 4_096**3 // 4:
        batch = (batch + 1) // 2
    while rows * cols * min(rows, cols) > 4_096**3 // 2:
        rows, cols = rows * 3 // 4, cols * 3 // 4
    noise = rng.choice((0.1, 0.3, 1.0))
    if op == "orthogonalise":
        return _orthogonalise(batch, rows, cols, rng.choice(("fp32", "bf16")), noise)
    return _muon(batch, rows, cols, rng.choice(("fp32", "bf16")), rng.choice(("fp32", "bf16")), noise)


def _tokens(case, gen):
    """Tokens spread over the vocabulary by their rank's logarithm, as words
    are: P(v) = log((v + 2) / (v + 1)) / log(V + 1)."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, dtype=torch.float64, device="cuda", generator=gen)
    ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    if case["masked"]:
        ids[torch.rand(T, device="cuda", generator=gen) < case["masked"]] = -1
    return ids.to(TYPES[case["ids"]])


def _gradients(case, gen, count):
    """`count` gradient-like stacks of matrices that share a few strong
    directions of falling strength, each with noise of its own."""
    b, m, n = case["batch"], case["rows"], case["cols"]
    r = max(2, min(m, n) // 16)
    u = torch.randn(b, m, r, device="cuda", generator=gen) / math.sqrt(m)
    v = torch.randn(b, r, n, device="cuda", generator=gen) / math.sqrt(n)
    strong = torch.bmm(u / torch.arange(1, r + 1, device="cuda"), v)
    level = case["noise"] * math.sqrt(math.pi**2 / 6) / math.sqrt(m * n)
    return [strong + level * torch.randn(b, m, n, device="cuda", generator=gen) for _ in range(count)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op == "lookup":
        state["tokens"] = _tokens(case, gen)
        state["table"] = (0.02 * torch.randn(case["V"], case["D"], device="cuda", generator=gen)).to(
            TYPES[case["table"]])
    elif op == "grad":
        state["tokens"] = _tokens(case, gen)
        state["grad"] = (0.01 * torch.randn(case["T"], case["D"], device="cuda", generator=gen)).to(
            TYPES[case["grad"]])
        if case["accumulate"]:
            state["out"] = (0.01 * torch.randn(case["V"], case["D"], device="cuda", generator=gen)).to(
                TYPES[case["out"]])
    elif op == "orthogonalise":
        state["x"] = _gradients(case, gen, 1)[0].to(TYPES[case["x"]])
    else:
        g, m = _gradients(case, gen, 2)
        state["grad"], state["momentum"] = g.to(TYPES[case["grad"]]), 8 * m
        state["weight"] = (0.02 * torch.randn(g.shape, device="cuda", generator=gen)).to(TYPES[case["weight"]])
    return state


# ------------------------------------------------------------ plain forms --
def _plain_lookup(tokens, table, scale, dtype):
    rows = table[tokens.clamp(min=0).long()].float() * scale
    return torch.where((tokens >= 0)[:, None], rows, 0.0).to(dtype)


def _plain_grad(tokens, grad, V, scale, dtype, out):
    rows = torch.where((tokens >= 0)[:, None], grad.float(), 0.0)
    total = torch.zeros(V, grad.shape[1], device=grad.device).index_add_(0, tokens.clamp(min=0).long(), rows) * scale
    return total.to(dtype) if out is None else out.copy_(out.float() + total)


def _plain_orthogonalise(x):
    a, b, c = COEFFICIENTS
    tall = x.shape[1] > x.shape[2]
    x = x.float()
    x = x.transpose(1, 2).contiguous() if tall else x
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x / (norm + EPS)).float()
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _plain_muon(weight, grad, momentum):
    g = grad.float()
    momentum.mul_(BETA).add_(g)
    o = _plain_orthogonalise(g + BETA * momentum)
    s = math.sqrt(max(1.0, weight.shape[1] / weight.shape[2]))
    weight.copy_(weight.float() * (1 - LR * DECAY) - LR * s * o)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import top_gradient_sparsification_amd as tgs
        if op == "lookup":
            return tgs.embedding_lookup(state["tokens"], state["table"], scale=case["scale"],
                                        out_dtype=TYPES[case["out"]])
        if op == "grad":
            return tgs.embedding_grad(state["tokens"], state["grad"], case["V"], scale=case["scale"],
                                      out_dtype=TYPES[case["out"]], out=state.get("out"),
                                      accumulate=case["accumulate"])
        if op == "orthogonalise":
            return tgs.newton_schulz(state["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        tgs.muon_step(state["weight"], state["grad"], state["momentum"], lr=LR, beta=BETA, nesterov=True,
                      weight_decay=DECAY, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return {"weight": state["weight"], "momentum": state["momentum"]}
    if op == "lookup":
        return _plain_lookup(state["tokens"], state["table"], case["scale"], TYPES[case["out"]])
    if op == "grad":
        return _plain_grad(state["tokens"], state["grad"], case["V"], case["scale"], TYPES[case["out"]],
                           state.get("out"))
    if op == "orthogonalise":
        return _plain_orthogonalise(state["x"]).to(state["x"].dtype)
    _plain_muon(state["weight"], state["grad"], state["momentum"])
    return {"weight": state["weight"], "momentum": state["momentum"]}


def work(case):
    op = case["op"]
    if op in ("lookup", "grad"):
        T, V, D = case["T"], case["V"], case["D"]
        places = T * (1 - case["masked"])
        v = np.arange(V, dtype=np.float64)
        p = np.log((v + 2) / (v + 1)) / math.log(V + 1)
        rows = float(-np.expm1(places * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())  # distinct tokens expected
        if op == "lookup":
            return {"bytes": T * BYTES[case["ids"]] + rows * D * BYTES[case["table"]] + T * D * BYTES[case["out"]],
                    "flops": T * D}
        moved = 2 * rows if case["accumulate"] else V
        return {"bytes": T * BYTES[case["ids"]] + places * D * BYTES[case["grad"]] + moved * D * BYTES[case["out"]],
                "flops": places * D}
    b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # A and A^2 are symmetric: half of each product suffices
    flops = b * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    if op == "orthogonalise":
        return {"bytes": b * m * n * 2 * BYTES[case["x"]], "flops": flops}
    return {"bytes": b * m * n * (BYTES[case["grad"]] + 2 * 4 + 2 * BYTES[case["weight"]]), "flops": flops}


# ------------------------------------------------------------------ exact --
def _polar(u):
    """The iteration in 64 bits, on the right and in nested form:
    X <- X (a + S (b + c S)) with S = X^T X over the shorter side."""
    a, b, c = COEFFICIENTS
    y = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + EPS)
    wide = y.shape[2] > y.shape[1]
    if wide:
        y = y.mT.contiguous()
    eye = torch.eye(y.shape[2], dtype=torch.float64, device=y.device)
    for _ in range(STEPS):
        s = torch.matmul(y.mT.contiguous(), y)
        y = torch.matmul(y, a * eye + torch.matmul(s, b * eye + c * s))
    return y.mT.contiguous() if wide else y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        t = st["tokens"].long()
        out = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
        real = torch.nonzero(t >= 0)[:, 0]
        out[real] = st["table"].index_select(0, t[real]).double() * case["scale"]
        return out
    if op == "grad":
        t = st["tokens"].long()
        real = torch.nonzero(t >= 0)[:, 0]
        order = real[torch.argsort(t[real], stable=True)]
        out = st["out"].double() if case["accumulate"] else torch.zeros(case["V"], case["D"], dtype=torch.float64,
                                                                       device="cuda")
        for part in order.split(8192):
            out.index_add_(0, t[part], st["grad"][part].double(), alpha=case["scale"])
        return out
    if op == "orthogonalise":
        return _polar(st["x"].double())
    g = st["grad"].double()
    m = BETA * st["momentum"].double() + g
    w = st["weight"].double()
    s = max(1.0, case["rows"] / case["cols"]) ** 0.5
    return {"weight": w - LR * (DECAY * w + s * _polar(g + BETA * m)), "momentum": m}
