"""The operators around a trained linear layer, as cases with a plain form.

- ``linear``:     y = act(x w^T + b) + r, with the pre-activation kept in full or in 8 bits
- ``backward``:   its gradients from checkpoints of x and of the pre-activation in 8 bits
- ``checkpoint``: an activation packed into 8 bits with a power-of-two scale per 32 channels,
                  and unpacked
- ``norm``:       h = x + r, y = h / rms(h) * g, with y in 8 bits as the next layer's checkpoint
- ``norm_back``:  its gradients

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
package's kernels.
"""
import math

import torch

own = False

GROUP = 32  # channels that share a scale
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------- cases

def _case(op, m, k, n=0, dtype="bf16", act="none", bias=True, res=False, save="none", name=None):
    c = {"op": op, "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias, "res": res, "save": save}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token through a BERT-base projection: the latency of one call
        _case("linear", 1, 768, 768, act="gelu", name="linear_one_token"),
        # a few tokens through an LLM MLP's up projection: the weight streamed once
        _case("linear", 8, 4096, 11008, act="silu", name="linear_few_tokens"),
        # BERT-base attention projection of a training batch, 32 x 512 tokens, residual added
        _case("linear", 16384, 768, 768, res=True, name="linear_bert_attn"),
        # LLM MLP up projection of a training batch, 8 x 2048 tokens; z is kept in 8 bits
        _case("linear", 16384, 4096, 11008, act="gelu_tanh", save="z8", name="linear_llm_up"),
        # the gradients of a tiny layer in float32: launches count
        _case("backward", 128, 64, 64, dtype="fp32", act="relu", name="backward_tiny"),
        # EfficientFormer-L1 last stage, 128 x 49 tokens
        _case("backward", 6272, 448, 1792, act="gelu", name="backward_effformer"),
        # the gradients of the LLM MLP's up projection
        _case("backward", 16384, 4096, 11008, act="gelu_tanh", name="backward_llm_up"),
        # one BERT sequence's activation packed and unpacked
        _case("checkpoint", 512, 768, name="checkpoint_sequence"),
        # the LLM MLP's hidden activation
        _case("checkpoint", 16384, 11008, name="checkpoint_llm_hidden"),
        # the norm of one token before a layer
        _case("norm", 1, 4096, res=True, name="norm_one_token"),
        # the norm of a training batch, writing the next layer's checkpoint
        _case("norm", 16384, 4096, res=True, save="y8", name="norm_llm"),
        # its gradients, with the residual stream's gradient added
        _case("norm_back", 16384, 4096, res=True, name="norm_back_llm"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "backward", "checkpoint", "norm", "norm_back"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    m = max(1, min(16384, int(_log(rng, 1, 16384))))
    wide = lambda hi: max(64, min(hi, 8 * int(_log(rng, 64, hi) / 8)))  # noqa: E731
    if op in ("linear", "backward"):
        k, n = (wide(4096), wide(11008)) if rng.random() < 0.5 else (wide(11008), wide(4096))
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        save = rng.choice(["none", "z", "z8"]) if op == "linear" else "none"
        return _case(op, m, k, n, dtype, act, rng.random() < 0.8, rng.random() < 0.5, save)
    k = wide(11008 if op == "checkpoint" else 8192)
    save = "y8" if op == "norm" and rng.random() < 0.5 else "none"
    return _case(op, m, k, 0, dtype, res=rng.random() < 0.7, save=save)


# -------------------------------------------------------------------------- plain parts

def _groups(x):
    """x [M, C] as [M, G, 32], zeros behind the last channel."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % GROUP)).unflatten(1, (-1, GROUP))


def _two_to(e, dtype=torch.float32):
    """2^e exactly, for exponents of normal numbers: its bits (pow is off by a rounding)."""
    if dtype == torch.float32:
        return ((e.to(torch.int32) + 127) << 23).view(torch.float32)
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _pack(x):
    """(q int8 [M, C], the scales' biased exponents uint8 [M, G]) of a float32 x."""
    t = _groups(x)
    amax = t.abs().amax(2, keepdim=True)
    m, e = torch.frexp(amax)
    e = torch.clamp(e - 7 + (m > 127 / 128), -126, 127)
    fine = torch.isfinite(amax)
    e = torch.where(fine, e, 0)
    q = torch.where(fine, torch.round(t * _two_to(-e)), 0)
    b = torch.where(fine, e + 127, 255)
    return q.flatten(1)[:, :x.shape[1]].to(torch.int8), b.squeeze(2).to(torch.uint8)


def _values(q, b):
    """What q and its scales stand for."""
    s = torch.where(b == 255, math.nan, _two_to(b.to(torch.int32).clamp(max=254) - 127))
    return (_groups(q.float()) * s.unsqueeze(2)).flatten(1)[:, :q.shape[1]]


def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# ------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    m, k, n = case["m"], case["k"], case["n"]

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * sd

    def activation(rows, cols):
        """Channels of different sizes, a few of them large, as layers' inputs are."""
        return (normal(rows, cols) * torch.exp(0.5 * normal(cols))).to(dt)

    s = {"case": case}
    if case["op"] == "linear":
        s["x"] = activation(m, k)
        s["w"] = normal(n, k, sd=k ** -0.5).to(dt)
        s["b"] = normal(n, sd=0.1).to(dt) if case["bias"] else None
        s["r"] = normal(m, n).to(dt) if case["res"] else None
    elif case["op"] == "backward":
        s["gy"] = normal(m, n, sd=0.01).to(dt)
        s["w"] = normal(n, k, sd=k ** -0.5).to(dt)
        s["x"] = _pack(activation(m, k).float())
        s["z"] = _pack(normal(m, n).to(dt).float()) if case["act"] != "none" else None
    elif case["op"] == "checkpoint":
        s["x"] = activation(m, k)
    elif case["op"] == "norm":
        s["x"] = activation(m, k)
        s["r"] = normal(m, k).to(dt) if case["res"] else None
        s["g"] = (1 + normal(k, sd=0.1)).to(dt)
    else:
        s["gy"] = normal(m, k, sd=0.01).to(dt)
        s["h"] = activation(m, k)
        s["g"] = (1 + normal(k, sd=0.1)).to(dt)
        s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
        s["gh"] = normal(m, k, sd=0.01).to(dt) if case["res"] else None
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)(case["op"], case, state)


def _own(op, case, s):
    from rank_compressed_backprop_amd import ops
    if op == "linear":
        y, z = ops.linear_forward(s["x"], s["w"], bias=s["b"], residual=s["r"], activation=case["act"],
                                  save=case["save"])
        if case["save"] == "z8":
            z = ops.checkpoint_unpack(z, torch.bfloat16)
        return {"y": y} if z is None else {"y": y, "z": z}
    if op == "backward":
        z = ops.Checkpoint8(*s["z"]) if s["z"] is not None else None
        gz, gb = ops.activation_backward(s["gy"], z, activation=case["act"], bias_grad=case["bias"])
        gx, gw = ops.linear_backward(gz, s["w"], ops.Checkpoint8(*s["x"]))
        return {"gx": gx, "gw": gw, "gb": gb} if case["bias"] else {"gx": gx, "gw": gw}
    if op == "checkpoint":
        c = ops.checkpoint_pack(s["x"])
        return {"x": ops.checkpoint_unpack(c, s["x"].dtype), "scale": c.scale}
    if op == "norm":
        out = ops.rmsnorm_forward(s["x"], s["g"], residual=s["r"], eps=EPS, y8=case["save"] == "y8")
        found = {"y": out.y, "rstd": out.rstd}
        if case["res"]:
            found["h"] = out.h
        if case["save"] == "y8":
            found["y8"] = ops.checkpoint_unpack(out.y8, torch.bfloat16)
        return found
    gx, gg = ops.rmsnorm_backward(s["gy"], s["h"], s["g"], s["rstd"], gh=s["gh"])
    return {"gx": gx, "gg": gg}


def _plain(op, case, s):
    dt = DT[case["dtype"]]
    if op == "linear":
        z = torch.matmul(s["x"].float(), s["w"].float().t())
        if case["bias"]:
            z = z + s["b"].float()
        y = _act(z, case["act"])
        if case["res"]:
            y = y + s["r"].float()
        if case["save"] == "z":
            return {"y": y.to(dt), "z": z.to(dt)}
        if case["save"] == "z8":
            return {"y": y.to(dt), "z": _values(*_pack(z)).to(torch.bfloat16)}
        return {"y": y.to(dt)}
    if op == "backward":
        gz = s["gy"].float()
        if s["z"] is not None:
            gz = gz * _act_slope(_values(*s["z"]), case["act"])
        gx = torch.matmul(gz, s["w"].float())
        gw = torch.matmul(gz.t(), _values(*s["x"]))
        if case["bias"]:
            return {"gx": gx.to(dt), "gw": gw.to(dt), "gb": gz.sum(0).to(dt)}
        return {"gx": gx.to(dt), "gw": gw.to(dt)}
    if op == "checkpoint":
        q, b = _pack(s["x"].float())
        return {"x": _values(q, b).to(dt), "scale": b}
    if op == "norm":
        h = s["x"]
        if case["res"]:
            h = (h.float() + s["r"].float()).to(dt)  # the residual stream is kept in its type
        f = h.float()
        rstd = torch.rsqrt((f * f).mean(1) + EPS)
        y = (f * rstd[:, None] * s["g"].float()).to(dt)
        found = {"y": y, "rstd": rstd}
        if case["res"]:
            found["h"] = h
        if case["save"] == "y8":
            found["y8"] = _values(*_pack(y.float())).to(torch.bfloat16)
        return found
    gy, h, g, rstd = s["gy"].float(), s["h"].float(), s["g"].float(), s["rstd"][:, None]
    t = gy * g
    gx = rstd * (t - h * rstd * rstd * (t * h).mean(1, keepdim=True))
    if case["res"]:
        gx = gx + s["gh"].float()
    return {"gx": gx.to(dt), "gg": (gy * h * rstd).sum(0).to(dt)}


def work(case):
    m, k, n = case["m"], case["k"], case["n"]
    e = 2 if case["dtype"] == "bf16" else 4
    eight = lambda c: m * c + m * (-(-c // GROUP))  # noqa: E731
    op = case["op"]
    if op == "linear":
        # z in 8 bits is also returned as the bf16 values that it stands for
        kept = {"none": 0, "z": m * n * e, "z8": 2 * m * n}[case["save"]]
        b = (m * k + n * k + m * n + (n if case["bias"] else 0) + (m * n if case["res"] else 0)) * e + kept
        return {"bytes": b, "flops": 2 * m * n * k}
    if op == "backward":
        b = (m * n + n * k + m * k + n * k + (n if case["bias"] else 0)) * e + eight(k)
        return {"bytes": b + (eight(n) if case["act"] != "none" else 0), "flops": 4 * m * n * k}
    if op == "checkpoint":
        return {"bytes": 2 * m * k * e + m * (-(-k // GROUP)), "flops": 4 * m * k}
    if op == "norm":
        b = (2 + (2 if case["res"] else 0)) * m * k * e + k * e + 4 * m
        return {"bytes": b + (2 * m * k if case["save"] == "y8" else 0), "flops": 6 * m * k}
    return {"bytes": (3 + (1 if case["res"] else 0)) * m * k * e + 2 * k * e + 4 * m, "flops": 10 * m * k}


# ------------------------------------------------------------------------------ 64 bits

def _slope64(z, name):
    """The activation's derivative by differentiating its definition."""
    with torch.enable_grad():
        z = z.detach().requires_grad_(True)
        if name == "relu":
            y = torch.where(z > 0, z, torch.zeros_like(z))
        elif name == "gelu":
            y = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        elif name == "gelu_tanh":
            y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif name == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z * 1.0
        return y.detach(), torch.autograd.grad(y.sum(), z)[0]


def _eight64(x):
    """x rounded to the nearest of the 255 multiples of its group's scale."""
    out = torch.zeros_like(x)
    for c in range(0, x.shape[1], GROUP):
        t = x[:, c:c + GROUP]
        top = t.abs().amax(1, keepdim=True).clamp(min=1e-300)
        e = torch.floor(torch.log2(top / 127)).clamp(-126, 126) - 1
        for _ in range(3):  # the first exponent whose 127 steps reach the largest value
            e = torch.where(top > 127 * _two_to(e, torch.float64), e + 1, e)
        s = _two_to(e.clamp(min=-126), torch.float64)
        out[:, c:c + GROUP] = torch.round(t / s) * s
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = s["x"].double() @ s["w"].double().T
        if case["bias"]:
            z += s["b"].double()
        y = _slope64(z, case["act"])[0]
        if case["res"]:
            y += s["r"].double()
        return {"y": y} if case["save"] == "none" else {"y": y, "z": z if case["save"] == "z" else _eight64(z)}
    if op == "backward":
        def wide(pair):
            q, b = pair
            s = _two_to(b.to(torch.int64) - 127, torch.float64)
            return q.double() * s.repeat_interleave(GROUP, 1)[:, :q.shape[1]]
        gz = s["gy"].double()
        if s["z"] is not None:
            gz = gz * _slope64(wide(s["z"]), case["act"])[1]
        found = {"gx": gz @ s["w"].double(), "gw": gz.T.contiguous() @ wide(s["x"])}
        if case["bias"]:
            found["gb"] = gz.sum(0)
        return found
    if op == "checkpoint":
        return {"x": _eight64(s["x"].double()), "scale": None}
    if op == "norm":
        h = s["x"]
        if case["res"]:
            h = (h.double() + s["r"].double()).to(h.dtype)
        t = h.double()
        rstd = 1 / torch.sqrt(torch.sum(t * t, 1) / case["k"] + EPS)
        y = t * rstd[:, None] * s["g"].double()
        found = {"y": y, "rstd": rstd}
        if case["res"]:
            found["h"] = s["x"].double() + s["r"].double()
        if case["save"] == "y8":
            found["y8"] = _eight64(y.to(DT[case["dtype"]]).double())
        return found
    with torch.enable_grad():  # y = h g rstd(h) with rstd's dependence on h written out
        h, g, gy, rstd = s["h"].double(), s["g"].double(), s["gy"].double(), s["rstd"].double()
        u = gy * g
        gx = u * rstd[:, None] - h * (rstd ** 3 / case["k"] * torch.sum(u * h, 1))[:, None]
        if case["res"]:
            gx = gx + s["gh"].double()
        return {"gx": gx, "gg": torch.einsum("mk,mk,m->k", gy, h, rstd)}
