"""Cases of the row operators between a model's hidden states and its losses:
what they compute in plain torch operations, the calls a user makes of the
library, and the work each cannot do without.

Three operators, each with its way back:

* ``norm`` / ``norm_grad``: layer norm over the last axis, y = (x - mean) rstd
  w + b with rstd = 1 / sqrt(var + eps), and the gradients of x, w and b.
* ``logprobs`` / ``logprobs_grad``: log p(token) of given tokens under
  p = softmax(logits / temperature), with the entropy and the top alternatives
  of each row, and the gradient of the logits.  A negative token is a masked
  place: zeros, and -1 for its alternatives.
* ``distill`` / ``distill_grad`` / ``distill_step``: KL(q || p) against a
  teacher's top logits, q = softmax(teacher / temperature) over the slots that
  hold an index, its gradient, and both in one call for places whose weights
  are known.  A place without any slot gives zeros.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "int32": torch.int32,
         "int64": torch.int64}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2, "int32": 4, "int64": 8}


def _norm(op, T, D, x, y, w):
    return {"op": op, "T": T, "D": D, "x": x, "y": y, "w": w}


def _logprobs(T, V, logits, pad=0, ids="int64", temperature=1.0, masked=0.0, banned=0.0, top=0, entropy=True):
    return {"op": "logprobs", "T": T, "V": V, "logits": logits, "pad": pad, "ids": ids, "temperature": temperature,
            "masked": masked, "banned": banned, "top": top, "entropy": entropy}


def _logprobs_grad(T, V, logits, pad=0, ids="int64", temperature=1.0, masked=0.0, banned=0.0, entropy=True):
    return dict(_logprobs(T, V, logits, pad, ids, temperature, masked, banned, 0, entropy), op="logprobs_grad")


def _distill(op, T, V, K, logits, teacher, pad=0, ids="int32", temperature=1.0, masked=0.0, banned=0.0):
    return {"op": op, "T": T, "V": V, "K": K, "logits": logits, "teacher": teacher, "pad": pad, "ids": ids,
            "temperature": temperature, "masked": masked, "banned": banned}


def listed():
    return [
        # one generated token's hidden state: latency
        dict(_norm("norm", 1, 4_096, "bf16", "bf16", "bf16"), name="norm one token"),
        # a training batch of long sequences
        dict(_norm("norm", 131_072, 2_048, "bf16", "bf16", "fp32"), name="norm long batch"),
        # a toy model's rows of odd width, all of them small: latency
        dict(_norm("norm_grad", 517, 131, "fp32", "fp32", "fp32"), name="norm grad small odd"),
        # a wide model's micro-batch, weights kept in fp32
        dict(_norm("norm_grad", 65_536, 4_096, "bf16", "bf16", "fp32"), name="norm grad long batch"),
        # a sampled token's log probability with twenty alternatives, as a server reports them: latency
        dict(_logprobs(1, 128_000, "bf16", temperature=0.7, banned=0.05, top=20), name="logprobs one token"),
        # rollouts scored under a policy: entropy, five alternatives, prompts masked
        dict(_logprobs(8_192, 64_000, "bf16", masked=0.05, top=5), name="logprobs long batch"),
        # a policy's gradient with an entropy bonus; fp32 logits of an odd vocabulary in padded rows
        dict(_logprobs_grad(1_021, 50_001, "fp32", pad=47, ids="int32", temperature=1.3, masked=0.1),
             name="logprobs grad odd padded"),
        # a training batch's cross entropy on the way back
        dict(_logprobs_grad(8_192, 32_000, "bf16", entropy=False), name="logprobs grad long batch"),
        # a few places against sixteen teacher's logits: latency
        dict(_distill("distill", 33, 32_000, 16, "fp32", "fp32", temperature=2.0), name="distill few places"),
        # a batch's loss as it is evaluated
        dict(_distill("distill", 8_192, 64_000, 64, "bf16", "fp16", masked=0.05), name="distill long batch"),
        # the loss's gradient for upstream values of each place, odd vocabulary, padded rows
        dict(_distill("distill_grad", 2_047, 50_001, 32, "fp16", "fp32", pad=47, ids="int64", temperature=2.0,
                      masked=0.1, banned=0.02), name="distill grad odd padded"),
        # a distilled model's training step over a large vocabulary
        dict(_distill("distill_step", 4_096, 128_000, 64, "bf16", "bf16", masked=0.02), name="distill step long batch"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "logprobs", "logprobs_grad", "distill", "distill_grad", "distill_step"))
    types = ("fp32", "bf16", "fp16")
    if op in ("norm", "norm_grad"):
        T, D = _between(rng, 1, 131_072), _between(rng, 2, 16_384)
        while T * D > 65_536 * 2_048:
            T = (T + 1) // 2
        x = rng.choice(types)
        return _norm(op, T, D, x, rng.choice((x, x, rng.choice(types))), rng.choice(types))
    T, V = _between(rng, 1, 16_384), _between(rng, 2, 128_000)
    while T * V > 2_048 * 64_000:
        T = (T + 1) // 2
    common = {"pad": rng.choice((0, 0, 1, 47)), "ids": rng.choice(("int32", "int64")),
              "temperature": rng.choice((1.0, 0.7, 2.0)), "masked": rng.choice((0.0, 0.05, 0.5)),
              "banned": rng.choice((0.0, 0.05)) if V >= 1_000 else 0.0}
    if op == "logprobs":
        return _logprobs(T, V, rng.choice(types), top=min(V, rng.choice((0, 1, 5, 20, 50))),
                         entropy=rng.random() < 0.5, **common)
    if op == "logprobs_grad":
        return _logprobs_grad(T, V, rng.choice(types), entropy=rng.random() < 0.5, **common)
    return _distill(op, T, V, min(_between(rng, 1, 256), max(1, V // 2)), rng.choice(types), rng.choice(types), **common)


def _logits(case, gen):
    """Rows like a language model's: normal scores, a few tokens of each row
    well above the others, banned tokens at -inf.  ``pad`` more columns belong
    to the rows' memory and not to the rows."""
    T, V = case["T"], case["V"]
    z = 2 * torch.randn(T, V, device="cuda", generator=gen)
    at = torch.randint(V, (T, 8), device="cuda", generator=gen)
    z.scatter_(1, at, 6 + 3 * torch.randn(T, 8, device="cuda", generator=gen))
    allowed = torch.rand(V, device="cuda", generator=gen) >= case["banned"]
    allowed[0] = True
    z.masked_fill_(~allowed, -math.inf)
    rows = torch.full((T, V + case["pad"]), 7.0, dtype=TYPES[case["logits"]], device="cuda")
    rows[:, :V] = z
    return rows[:, :V], torch.nonzero(allowed)[:, 0], z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state, T = case["op"], {"case": case}, case["T"]
    if op in ("norm", "norm_grad"):
        D, w = case["D"], TYPES[case["w"]]
        # hidden states: columns of unlike size and mean, rows of unlike size
        columns = torch.exp(0.5 * torch.randn(D, device="cuda", generator=gen))
        x = torch.randn(T, D, device="cuda", generator=gen) * columns + 0.2 * torch.randn(D, device="cuda", generator=gen)
        x = (x * torch.exp(0.3 * torch.randn(T, 1, device="cuda", generator=gen))).to(TYPES[case["x"]])
        state["x"] = x
        state["weight"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).to(w)
        state["bias"] = (0.1 * torch.randn(D, device="cuda", generator=gen)).to(w)
        if op == "norm_grad":
            state["grad"] = (0.1 * torch.randn(T, D, device="cuda", generator=gen)).to(TYPES[case["y"]])
            # what the forward pass left
            mean, rstd = [], []
            for part in x.split(8192):
                part = part.double()
                mean.append(part.mean(1))
                rstd.append(1 / (part.var(1, correction=0) + EPS).sqrt())
            state["mean"], state["rstd"] = torch.cat(mean).float(), torch.cat(rstd).float()
        return state
    state["logits"], allowed, z = _logits(case, gen)
    masked = torch.rand(T, device="cuda", generator=gen) < case["masked"]
    if op in ("logprobs", "logprobs_grad"):
        tokens = allowed[torch.randint(allowed.numel(), (T,), device="cuda", generator=gen)]
        state["tokens"] = torch.where(masked, -1, tokens).to(TYPES[case["ids"]])
        if op == "logprobs_grad":
            state["grad"] = torch.randn(T, device="cuda", generator=gen)
            state["grad_entropy"] = 0.1 * torch.randn(T, device="cuda", generator=gen) if case["entropy"] else None
    else:
        K = case["K"]
        near = z.add_(torch.randn(z.shape, device="cuda", generator=gen))
        at = torch.topk(near, K, dim=1)
        slots = torch.randint(max(1, K // 2), K + 1, (T, 1), device="cuda", generator=gen)  # teachers return K at most
        slots[masked] = 0
        empty = torch.arange(K, device="cuda") >= slots
        state["indices"] = at.indices.masked_fill(empty, -1).to(TYPES[case["ids"]])
        state["teacher"] = at.values.to(TYPES[case["teacher"]])
        if op != "distill":
            state["weights"] = torch.rand(T, device="cuda", generator=gen)
    if op in ("logprobs_grad", "distill_grad"):  # what the forward pass left
        tau, top, logsum, entropy = case["temperature"], [], [], []
        for part in state["logits"].split(max(1, (1 << 27) // case["V"])):
            part = part.double()
            m = part.max(1).values
            d = (part - m[:, None]) / tau
            s = d.exp().sum(1)
            top.append(m)
            logsum.append(s.log())
            entropy.append(s.log() - (d.exp() * d.clamp(min=-1e4)).sum(1) / s)
        state["stats"] = torch.stack([torch.cat(top), torch.cat(logsum)], 1).float()
        if case.get("entropy"):
            state["entropy"] = torch.cat(entropy).float()
            state["stats"][masked], state["entropy"][masked] = 0, 0
    return state


# ------------------------------------------------------------ plain forms --
def _plain_norm(st, dtype):
    x = st["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return (d * rstd * st["weight"].float() + st["bias"].float()).to(dtype)


def _plain_norm_grad(st):
    x, g, w = st["x"].float(), st["grad"].float(), st["weight"].float()
    hat = (x - st["mean"][:, None]) * st["rstd"][:, None]
    gw = g * w
    gx = (gw - gw.mean(1, keepdim=True) - hat * (gw * hat).mean(1, keepdim=True)) * st["rstd"][:, None]
    return {"x": gx.to(st["x"].dtype), "weight": (g * hat).sum(0).to(st["weight"].dtype),
            "bias": g.sum(0).to(st["weight"].dtype)}


def _plain_logprobs(st, case):
    tokens, real = st["tokens"].long(), st["tokens"] >= 0
    x = st["logits"].float()
    top = x.max(1, keepdim=True).values
    d = (x - top) / case["temperature"]
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    logs = torch.log(s)
    lp = d.gather(1, tokens.clamp(min=0)[:, None]) - logs
    out = {"logprobs": torch.where(real, lp[:, 0], 0.0)}
    if case["entropy"]:
        h = logs[:, 0] - torch.where(e > 0, e * d, 0.0).sum(1) / s[:, 0]
        out["entropy"] = torch.where(real, h, 0.0)
    if case["top"]:
        places = []
        x = x.clone()
        for _ in range(case["top"]):
            at = x.max(1, keepdim=True).indices  # of equal ones the first
            places.append(at)
            x.scatter_(1, at, -math.inf)
        at = torch.cat(places, 1)
        out["top_logprobs"] = torch.where(real[:, None], d.gather(1, at) - logs, 0.0)
        out["top_indices"] = torch.where(real[:, None], at, -1).int()
    return out


def _plain_probabilities(st, case):
    """log p and p of every entry, from what the forward pass left."""
    lp = (st["logits"].float() - st["stats"][:, :1]) / case["temperature"] - st["stats"][:, 1:]
    return lp, torch.exp(lp)


def _plain_logprobs_grad(st, case):
    tokens, real = st["tokens"].long(), (st["tokens"] >= 0)[:, None]
    lp, p = _plain_probabilities(st, case)
    g = st["grad"][:, None]
    out = -g * p
    if case["entropy"]:
        out -= torch.where(p > 0, st["grad_entropy"][:, None] * p * (lp + st["entropy"][:, None]), 0.0)
    out.scatter_add_(1, tokens.clamp(min=0)[:, None], g)
    return torch.where(real, out / case["temperature"], 0.0).to(st["logits"].dtype)


def _plain_teacher(st, case):
    """(q, log q, index) of the slots; empty ones have q = 0."""
    at = st["indices"].long()
    t = torch.where(at >= 0, st["teacher"].float() / case["temperature"], -math.inf)
    t = t - t.max(1, keepdim=True).values.clamp(min=-1e30)
    e = torch.exp(t)
    s = e.sum(1, keepdim=True).clamp(min=1e-30)
    return e / s, torch.where(e > 0, t - torch.log(s), 0.0), at.clamp(min=0)


def _plain_distill(st, case):
    q, lq, at = _plain_teacher(st, case)
    x = st["logits"].float()
    d = (x - x.max(1, keepdim=True).values) / case["temperature"]
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    terms = q * (lq - (d.gather(1, at) - torch.log(s)))
    return torch.where(q > 0, terms, 0.0).sum(1), e / s, q, at


def _plain_distill_grad(p, q, at, scale, dtype):
    out = p.mul_(q.sum(1, keepdim=True)).scatter_add_(1, at, -q)
    return out.mul_(scale[:, None]).to(dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import top_gradient_sparsification_amd as tgs
        if op == "norm":
            return tgs.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS, out_dtype=TYPES[case["y"]])
        if op == "norm_grad":
            gx, gw, gb = tgs.layer_norm_grad(state["grad"], state["x"], state["mean"], state["rstd"], state["weight"])
            return {"x": gx, "weight": gw, "bias": gb}
        if op == "logprobs":
            r = tgs.token_logprobs(state["logits"], state["tokens"], temperature=case["temperature"], top=case["top"],
                                   entropy=case["entropy"])
            out = {"logprobs": r.logprobs}
            if case["entropy"]:
                out["entropy"] = r.entropy
            if case["top"]:
                out["top_logprobs"], out["top_indices"] = r.top_logprobs, r.top_indices
            return out
        if op == "logprobs_grad":
            return tgs.token_logprobs_grad(state["logits"], state["tokens"], state["stats"], state["grad"],
                                           entropy=state.get("entropy"), grad_entropy=state["grad_entropy"],
                                           temperature=case["temperature"])
        given = state["logits"], state["indices"], state["teacher"]
        if op == "distill":
            return tgs.distillation_loss(*given, temperature=case["temperature"])
        if op == "distill_grad":
            return tgs.distillation_grad(*given, state["stats"], state["weights"], temperature=case["temperature"])
        loss, grad = tgs.distillation_loss_and_grad(*given, weights=state["weights"], temperature=case["temperature"])
        return {"loss": loss, "grad": grad}
    if op == "norm":
        return _plain_norm(state, TYPES[case["y"]])
    if op == "norm_grad":
        return _plain_norm_grad(state)
    if op == "logprobs":
        return _plain_logprobs(state, case)
    if op == "logprobs_grad":
        return _plain_logprobs_grad(state, case)
    if op == "distill":
        return _plain_distill(state, case)[0]
    dtype = state["logits"].dtype
    if op == "distill_grad":
        p = _plain_probabilities(state, case)[1]
        q, _, at = _plain_teacher(state, case)
        return _plain_distill_grad(p, q, at, state["weights"] / case["temperature"], dtype)
    loss, p, q, at = _plain_distill(state, case)
    return {"loss": loss, "grad": _plain_distill_grad(p, q, at, state["weights"] / case["temperature"], dtype)}


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_grad"):
        D, x, y, w = case["D"], BYTES[case["x"]], BYTES[case["y"]], BYTES[case["w"]]
        if op == "norm":
            return {"bytes": T * D * (x + y) + 2 * D * w, "flops": 8 * T * D}
        return {"bytes": T * D * (2 * x + y) + 8 * T + 3 * D * w, "flops": 14 * T * D}
    V, z, real = case["V"], BYTES[case["logits"]], T * (1 - case["masked"])
    if op == "logprobs":
        n = 1 + case["entropy"] + 2 * case["top"]
        return {"bytes": real * V * z + T * (BYTES[case["ids"]] + 4 * n), "flops": real * V * (4 + 2 * case["entropy"])}
    if op == "logprobs_grad":
        n = 3 + 2 * case["entropy"]
        return {"bytes": (real + T) * V * z + T * (BYTES[case["ids"]] + 4 * n),
                "flops": real * V * (4 + 3 * case["entropy"])}
    teacher = T * case["K"] * (BYTES[case["ids"]] + BYTES[case["teacher"]])
    if op == "distill":
        return {"bytes": real * V * z + teacher + 4 * T, "flops": real * V * 4}
    return {"bytes": (real + T) * V * z + teacher + 12 * T, "flops": real * V * (4 if op == "distill_grad" else 6)}


# ------------------------------------------------------------------ exact --
def _exact_norm(st, case, T, D):
    w, b = st["weight"].double(), st["bias"].double()
    if case["op"] == "norm":
        out = torch.empty(T, D, dtype=torch.float64, device="cuda")
        for i in range(0, T, 4096):
            x = st["x"][i:i + 4096].double()
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            out[i:i + 4096] = torch.addcmul(b, (x - mean) * torch.rsqrt(var + EPS), w)
        return out
    gx = torch.empty(T, D, dtype=torch.float64, device="cuda")
    gw, gb = torch.zeros_like(w), torch.zeros_like(w)
    for i in range(0, T, 4096):
        x, g = st["x"][i:i + 4096].double(), st["grad"][i:i + 4096].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        r = torch.rsqrt(var + EPS)
        h = (x - mean) * r
        a = g * w
        gx[i:i + 4096] = r / D * (D * a - a.sum(1, keepdim=True) - h * (a * h).sum(1, keepdim=True))
        gw += torch.linalg.vecdot(g, h, dim=0)
        gb += g.sum(0)
    return {"x": gx, "weight": gw, "bias": gb}


def exact(case, seed):
    st = prepare(case, seed)
    op, T, tau = case["op"], case["T"], case.get("temperature")
    if op in ("norm", "norm_grad"):
        return _exact_norm(st, case, T, case["D"])
    V = case["V"]
    rows = max(1, (1 << 27) // V)
    kept = {}

    def keep(name, value):
        kept.setdefault(name, []).append(value)

    for i in range(0, T, rows):
        z = st["logits"][i:i + rows].double() / tau
        n = z.shape[0]
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        if op in ("logprobs", "logprobs_grad"):
            t = st["tokens"][i:i + rows].long()
            on = (t >= 0).double()[:, None]
            line = torch.arange(n, device="cuda")
            h = -torch.xlogy(lp.exp(), lp.exp()).sum(1, keepdim=True)
            if op == "logprobs":
                keep("logprobs", lp[line, t.clamp(min=0)] * on[:, 0])
                if case["entropy"]:
                    keep("entropy", (h * on)[:, 0])
                if case["top"]:
                    keep("top_indices", torch.full((n, case["top"]), -1, dtype=torch.int32, device="cuda"))
                    keep("top_logprobs", torch.zeros(n, case["top"], dtype=torch.float64, device="cuda"))
                    for j in range(0, n, 256):
                        part = st["logits"][i + j:min(i + j + 256, i + n)].float()
                        # a stable order: equal scores by index
                        order = torch.argsort(part, dim=1, descending=True, stable=True)[:, :case["top"]]
                        live = t[j:j + 256] >= 0
                        kept["top_indices"][-1][j:j + 256][live] = order[live].int()
                        kept["top_logprobs"][-1][j:j + 256][live] = lp[j:j + 256].gather(1, order)[live]
                continue
            g = st["grad"][i:i + rows].double()[:, None]
            d = torch.zeros_like(lp)
            d[line, t.clamp(min=0)] = 1
            d = g * (d - lp.exp())
            if case["entropy"]:
                p = lp.exp()
                d -= st["grad_entropy"][i:i + rows].double()[:, None] * (torch.xlogy(p, p) + p * h)
            keep("grad", d * on / tau)
            continue
        t = st["teacher"][i:i + rows].double() / tau
        at = st["indices"][i:i + rows].long()
        q = torch.softmax(t.masked_fill(at < 0, -math.inf), 1).nan_to_num(0.0)  # places without a slot
        if op != "distill_grad":
            keep("loss", (torch.xlogy(q, q) - torch.where(q > 0, q * lp.gather(1, at.clamp(min=0)), 0.0)).sum(1))
        if op != "distill":
            d = lp.exp() * (q.sum(1, keepdim=True) > 0.5)
            d = d.index_put((torch.arange(n, device="cuda")[:, None].expand_as(at), at.clamp(min=0)), -q, accumulate=True)
            keep("grad", d * (st["weights"][i:i + rows].double() / tau)[:, None])
    out = {name: torch.cat(parts) for name, parts in kept.items()}
    return out["grad"] if op in ("logprobs_grad", "distill_grad") else out["loss"] if op == "distill" else out
