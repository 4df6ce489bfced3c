"""The operators at the two ends of a language model's training step, as cases with a plain form.

- ``logprobs``:      log probabilities of given tokens from logits, with the log of the sum, the
                     entropy and the most likely alternatives
- ``logprobs_back``: the logits' gradient, from gradients of the log probability and the entropy
- ``embed``:         rows of a table looked up by token, scaled
- ``embed_back``:    the table's gradient: rows of the gradient summed by token
- ``clip``:          the norm over all gradients of a model, and the gradients scaled by it
- ``norm``:          the norm alone

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
package's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100  # the target of a token without a loss
PAD = 0        # the token that fills a batch up: its embedding gets no gradient
CLIP_EPS = 1e-6


# ------------------------------------------------------------------------------- cases

def _logits(op, m, v, dtype="bf16", top=0, masked=0.0, ent=False, name=None):
    c = {"op": op, "m": m, "v": v, "dtype": dtype, "top": top, "masked": masked, "ent": ent}
    return c | {"name": name} if name else c


def _embed(op, m, v, c, dtype="bf16", name=None):
    c = {"op": op, "m": m, "v": v, "c": c, "dtype": dtype}
    return c | {"name": name} if name else c


def _grads(op, layers, c, h, v, dtype="bf16", out="same", name=None):
    c = {"op": op, "layers": layers, "c": c, "h": h, "v": v, "dtype": dtype, "out": out}
    return c | {"name": name} if name else c


def listed():
    return [
        # the next token of one sequence, with its alternatives: the latency of one call
        _logits("logprobs", 1, 32000, top=5, name="logprobs_one_token"),
        # the next tokens of a batch that is served, part of the vocabulary not allowed
        _logits("logprobs", 64, 128000, "fp32", top=20, masked=0.25, name="logprobs_serving"),
        # the loss and accuracy of a BERT-base batch, 32 x 512 tokens; rows of 61044 bytes, so that
        # three of four start off a 16-byte border
        _logits("logprobs", 16384, 30522, top=1, name="logprobs_bert"),
        # the loss of an LLM's batch, 4 x 2048 tokens
        _logits("logprobs", 8192, 128000, name="logprobs_llm"),
        # the gradient of a small model's policy, entropy kept up by a bonus; odd rows
        _logits("logprobs_back", 300, 1001, "fp32", ent=True, name="logprobs_back_small"),
        # the gradient of the LLM's loss
        _logits("logprobs_back", 8192, 128000, name="logprobs_back_llm"),
        # the tokens of a step of serving: the latency of one call
        _embed("embed", 8, 128000, 4096, name="embed_serving"),
        # a training batch of 8 x 2048 tokens
        _embed("embed", 16384, 128000, 4096, name="embed_llm"),
        # the gradient of a small table in float32: launches count
        _embed("embed_back", 64, 1000, 64, "fp32", name="embed_back_small"),
        # the gradient of a large table
        _embed("embed_back", 16384, 32000, 4096, name="embed_back_llm"),
        # a small model's 28 gradients in float32: launches count
        _grads("clip", 2, 64, 256, 1000, "fp32", name="clip_small"),
        # four layers of an LLM with its embedding, 0.94 G values
        _grads("clip", 4, 4096, 11008, 32000, name="clip_llm"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_back", "embed", "embed_back", "clip", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    size = 2 if dtype == "bf16" else 4
    if op in ("logprobs", "logprobs_back"):
        v = _log(rng, 256, 128000)
        m = _log(rng, 1, min(16384, 8192 * 128000 * 2 // (v * size)))
        top = rng.choice([0, 0, 1, 5, 20, 32]) if op == "logprobs" else 0
        return _logits(op, m, v, dtype, top, rng.choice([0.0, 0.0, 0.5]), op == "logprobs_back" and rng.random() < 0.5)
    if op in ("embed", "embed_back"):
        v, c = _log(rng, 256, 128000), 8 * _log(rng, 8, 512)
        m = _log(rng, 1, 16384)
        if op == "embed_back":  # (the dense gradient of the largest listed case)
            v = min(v, 32000 * 4096 * 2 // (c * size))
        return _embed(op, m, v, c, dtype)
    c = 8 * _log(rng, 8, 512)
    return _grads(op, rng.randint(1, 3 if c > 1024 else 12), c, 8 * _log(rng, 8, 640), _log(rng, 256, 32000), dtype,
                  rng.choice(["same", "same", "fp32"]) if op == "clip" else "same")


def _shapes(case):
    """The gradients of a model: an embedding, and in each layer four projections, two layers of an
    MLP, their biases and two norms."""
    c, h = case["c"], case["h"]
    layer = [(c, c)] * 4 + [(h, c), (c, h), (h,), (c,), (c,), (c,), (4 * c,), (1,), (1, c)]
    return [(case["v"], c)] + layer * case["layers"] + [(c,)]


# ------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    op = case["op"]

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * sd

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    if op in ("logprobs", "logprobs_back"):
        m, v = case["m"], case["v"]
        column = normal(v, sd=1.5)  # frequent tokens have larger logits
        allowed = torch.arange(v, device="cuda")
        if case["masked"]:
            mask = uniform(v) < case["masked"]
            mask[::4] = False
            allowed = allowed[~mask]
            column = torch.where(mask, -math.inf, column)
        z = torch.randn(m, v, generator=g, device="cuda")
        z = z.mul_(2).add_(column)
        z = z.add_(normal(m, 1, sd=3.0))
        t = allowed[torch.randint(allowed.numel(), (m,), generator=g, device="cuda")]
        rows = torch.arange(m, device="cuda")
        z[rows, t] += torch.where(uniform(m) < 0.5, 9.0, 0.0)  # what the model has learnt
        s["z"] = z.to(dt)
        s["t"] = torch.where(uniform(m) < 0.1, IGNORE, t) if m > 16 else t
        if op == "logprobs_back":
            s["g"] = normal(m, sd=1.0 / m)
            s["gh"] = normal(m, sd=0.01 / m) if case["ent"] else None
            # what the forward pass has left
            top, ls, h = (torch.empty(m, device="cuda") for _ in range(3))
            for a, b in _row_blocks(m, v):
                f = s["z"][a:b].double()
                top[a:b] = f.amax(1)
                f = f - f.amax(1, keepdim=True)
                e = torch.exp(f)
                ls[a:b] = torch.log(e.sum(1))
                h[a:b] = torch.log(e.sum(1)) - torch.where(e > 0, e * f, 0).sum(1) / e.sum(1)
            s["stats"], s["h"] = torch.stack((top, ls), 1).contiguous(), h
    elif op in ("embed", "embed_back"):
        m, v, c = case["m"], case["v"], case["c"]
        # a few tokens make up much of a text
        t = (torch.exp(uniform(m) * math.log(v)) - 1).long().clamp(0, v - 1)
        s["t"] = torch.where(uniform(m) < 0.05, PAD, t)
        s["scale"] = c ** 0.5
        if op == "embed":
            s["w"] = normal(v, c, sd=c ** -0.5).to(dt)
        else:
            s["gy"] = normal(m, c, sd=0.01).to(dt)
    else:
        shapes = _shapes(case)
        n = sum(math.prod(p) for p in shapes)
        s["g"] = [normal(*p, sd=2.5 * n ** -0.5).to(dt) for p in shapes]
        if op == "clip":
            # the optimizer's buffer: each gradient in its place, at a multiple of 64 values
            ends = [0]
            for p in shapes:
                ends.append(ends[-1] + -(-math.prod(p) // 64) * 64)
            s["flat"] = torch.zeros(ends[-1], device="cuda", dtype=dt if case["out"] == "same" else torch.float32)
            s["out"] = [s["flat"][a:a + math.prod(p)].view(p) for a, p in zip(ends, shapes)]
            s["max"] = 1.0
    return s


def _row_blocks(m, v):
    """Rows in blocks of about 2^25 values."""
    step = max(1, (1 << 25) // v)
    return [(a, min(m, a + step)) for a in range(0, m, step)]


# --------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)(case["op"], case, state)


def _own(op, case, s):
    from rank_compressed_backprop_amd import ops
    if op == "logprobs":
        out = ops.token_logprobs(s["z"], s["t"], top=case["top"], ignore=IGNORE)
        found = {"logp": out.logp, "lse": out.lse, "entropy": out.entropy}
        return found | ({"top": out.top_logp, "index": out.top_index} if case["top"] else {})
    if op == "logprobs_back":
        return ops.token_logprobs_backward(s["z"], s["t"], s["stats"], g_logp=s["g"], g_entropy=s["gh"],
                                           entropy=s["h"], ignore=IGNORE)
    if op == "embed":
        return ops.embedding_forward(s["t"], s["w"], scale=s["scale"])
    if op == "embed_back":
        return ops.embedding_backward(s["gy"], s["t"], case["v"], scale=s["scale"], padding=PAD)
    if op == "norm":
        return ops.grad_norm(s["g"])
    norm = ops.clip_grads(s["g"], s["max"], out=s["out"])
    return {"norm": norm, "g": s["flat"]}


def _plain(op, case, s):
    dt = DT[case["dtype"]]
    if op == "logprobs":
        z, t = s["z"].float(), s["t"]
        at = t.clamp(min=0)[:, None]
        top = z.amax(1, keepdim=True)
        d = z - top
        e = torch.exp(d)
        total = e.sum(1)
        ls = torch.log(total)
        logp = torch.where(t == IGNORE, 0.0, d.gather(1, at)[:, 0] - ls)
        entropy = ls - torch.where(e > 0, e * d, 0.0).sum(1) / total
        found = {"logp": logp, "lse": top[:, 0] + ls, "entropy": entropy}
        if case["top"]:
            del e
            column = torch.arange(case["v"], device="cuda", dtype=torch.int32)
            values, places = [], []
            for _ in range(case["top"]):  # the largest that is left, the lowest place of equal ones
                best = d.amax(1, keepdim=True)
                place = torch.where(d == best, column, case["v"]).amin(1).long()
                values.append(best[:, 0] - ls)
                places.append(place)
                d.scatter_(1, place[:, None], math.nan)
                d = torch.where(d == d, d, -math.inf)
            found["top"], found["index"] = torch.stack(values, 1), torch.stack(places, 1)
        return found
    if op == "logprobs_back":
        z, t = s["z"].float(), s["t"]
        seen = t != IGNORE
        g = torch.where(seen, s["g"], 0.0)[:, None]
        logp = (z - s["stats"][:, :1]) - s["stats"][:, 1:]
        p = torch.exp(logp)
        gz = -g * p
        if s["gh"] is not None:
            gz = gz - torch.where(p > 0, s["gh"][:, None] * p * (logp + s["h"][:, None]), 0.0)
        gz.scatter_add_(1, t.clamp(min=0)[:, None], g)
        return gz.to(dt)
    if op == "embed":
        return (s["w"][s["t"]].float() * s["scale"]).to(dt)
    if op == "embed_back":
        gy = torch.where((s["t"] == PAD)[:, None], 0.0, s["gy"].float())
        gw = torch.zeros(case["v"], case["c"], device="cuda")
        gw.index_add_(0, s["t"], gy)
        return (gw * s["scale"]).to(dt)
    total = 0.0
    for x in s["g"]:
        total = total + x.double().square().sum()
    norm = torch.sqrt(total).float()
    if op == "norm":
        return norm
    factor = torch.clamp(s["max"] / (norm + CLIP_EPS), max=1.0)
    for x, y in zip(s["g"], s["out"]):
        y.copy_(x.float() * factor)
    return {"norm": norm, "g": s["flat"]}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "logprobs":
        m, v, k = case["m"], case["v"], case["top"]
        return {"bytes": m * v * e + m * (8 + 12 + 12 * k), "flops": 6 * m * v}
    if op == "logprobs_back":
        m, v = case["m"], case["v"]
        return {"bytes": 2 * m * v * e + m * (8 + 12 + (8 if case["ent"] else 0)), "flops": (8 if case["ent"] else 4) * m * v}
    if op == "embed":
        m, v, c = case["m"], case["v"], case["c"]
        return {"bytes": (m + min(m, v)) * c * e + 8 * m, "flops": m * c}
    if op == "embed_back":
        m, v, c = case["m"], case["v"], case["c"]
        return {"bytes": (m + v) * c * e + 8 * m, "flops": m * c + min(m, v) * c}
    n = sum(math.prod(p) for p in _shapes(case))
    if op == "norm":
        return {"bytes": n * e + 4, "flops": 2 * n}
    return {"bytes": n * (e + (e if case["out"] == "same" else 4)) + 4, "flops": 3 * n}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("logprobs", "logprobs_back"):
        parts = []
        for a, b in _row_blocks(case["m"], case["v"]):
            z, t = s["z"][a:b].double(), s["t"][a:b]
            seen = t != IGNORE
            lse = torch.logsumexp(z, 1)
            logp = z - lse[:, None]
            p = torch.softmax(z, 1)
            entropy = -torch.xlogy(p, p).sum(1)
            rows = torch.arange(b - a, device="cuda")
            mine = torch.where(seen, logp[rows, torch.where(seen, t, 0)], 0.0)
            if op == "logprobs":
                found = {"logp": mine, "lse": lse, "entropy": entropy}
                if case["top"]:
                    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]
                    found["top"], found["index"] = logp[rows[:, None], order], order
                parts.append(found)
                continue
            # d logp_t / d z_j = [j = t] - p_j;  d H / d z_j = -p_j (log p_j + H)
            gz = torch.zeros_like(z)
            gz[rows, torch.where(seen, t, 0)] = 1.0
            gz = (gz - p) * (s["g"][a:b].double() * seen)[:, None]
            if s["gh"] is not None:
                gz -= s["gh"][a:b].double()[:, None] * (torch.xlogy(p, p) + p * entropy[:, None])
            parts.append(gz)
        if op == "logprobs":
            return {k: torch.cat([f[k] for f in parts]) for k in parts[0]}
        return torch.cat(parts)
    if op == "embed":
        return torch.stack([s["w"][i] for i in s["t"].tolist()]).double() * s["scale"]
    if op == "embed_back":
        order = torch.argsort(s["t"], stable=True)
        tokens, counts = torch.unique_consecutive(s["t"][order], return_counts=True)
        gw = torch.zeros(case["v"], case["c"], dtype=torch.float64, device="cuda")
        for v, rows in zip(tokens.tolist(), torch.split(order, counts.tolist())):
            if v != PAD:
                gw[v] = s["gy"][rows].double().sum(0) * s["scale"]
        return gw
    norm = math.sqrt(math.fsum(torch.dot(x, x).item() for x in (y.double().flatten() for y in s["g"])))
    found = torch.tensor(norm, dtype=torch.float64)
    if op == "norm":
        return found.cuda()
    flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for x in s["g"]:
        flat[at:at + x.numel()] = x.double().flatten() * min(1.0, s["max"] / (norm + CLIP_EPS))
        at += -(-x.numel() // 64) * 64
    return {"norm": found.cuda(), "g": flat}
