"""What is measured of the layer norm and the gated feed-forward block.

The two operators make the residual block z + FFN(LN(z)) of a network that predicts a matrix's coefficients from
features of the grid cells, one token a cell: a 64 x 64 grid has 4,096 tokens, a 128 x 128 grid 16,384 and a
1000 x 1000 grid 1,000,000.  A case is one forward call ("forward": inference) or a training step's forward and
backward call ("train").

    layer norm    y = (x - mean x) / sqrt(var x + eps) * w + b, over rows of `width`
    gated FFN     y = (act(x Wg^T + bg) * (x Wu^T + bu)) Wo^T + bo, `width` -> `hidden` -> `out`;
                  w_in stacks Wg over Wu, [2 hidden, width]; w_out is Wo, [out, hidden]
"""
import math

import torch

own = False

EPS = 1e-5
ROOT_2 = math.sqrt(2.0)
TANH_A, TANH_B = math.sqrt(2.0 / math.pi), 0.044715
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def ln(name, mode, rows, width, dtype, params=None):
    return {"name": name, "op": "layer_norm", "mode": mode, "rows": rows, "width": width, "dtype": dtype,
            "params": params or dtype}


def ffn(name, mode, rows, width, hidden, dtype, act="silu", bias=True, out=None):
    return {"name": name, "op": "gated_ffn", "mode": mode, "rows": rows, "width": width, "hidden": hidden,
            "out": out or width, "dtype": dtype, "act": act, "bias": bias}


def listed():
    return [
        # one query point answered by a trained network: latency
        ln("ln one row", "forward", 1, 1024, "bf16"),
        # a step on a 64 x 64 grid in full precision, as the solver's own data
        ln("ln 64x64 fp32 train", "train", 4096, 256, "fp32"),
        # every cell of the 1000 x 1000 grid, narrow rows
        ln("ln 1000x1000 train", "train", 1_000_000, 64, "bf16"),
        # an odd number of cells and a width that no vector load divides, parameters kept in 32 bits
        ln("ln odd train", "train", 5003, 1001, "fp16", params="fp32"),
        # one query point through the block: the weights are read once and little else
        ffn("ffn one token", "forward", 1, 1024, 4096, "bf16"),
        # a handful of probes (sensor places) at once, no biases
        ffn("ffn 13 tokens", "forward", 13, 768, 2048, "fp16", act="gelu_tanh", bias=False),
        # inference on every cell of the 1000 x 1000 grid with a narrow network
        ffn("ffn 1000x1000 narrow", "forward", 1_000_000, 64, 256, "bf16"),
        # training on a 64 x 64 grid, in the solver's single precision and in 16 bits
        ffn("ffn 64x64 fp32 train", "train", 4096, 256, 1024, "fp32", act="gelu"),
        ffn("ffn 64x64 train", "train", 4096, 256, 1024, "bf16", act="gelu"),
        # sizes that divide nothing: 2,049 tokens, 250 -> 683 -> 131
        ffn("ffn odd train", "train", 2049, 250, 683, "fp16", act="relu", out=131),
        # inference of a wide network on a 128 x 128 grid
        ffn("ffn 128x128 wide", "forward", 16384, 1024, 4096, "bf16", bias=False),
        # training the wide network on a batch of two 128 x 128 grids: the largest
        ffn("ffn 2x128x128 wide train", "train", 32768, 1024, 4096, "bf16"),
    ]


MOST_FLOPS = 18 * 32768 * 1024 * 4096  # the largest listed case's
MOST_BYTES = 4 * 1_000_000 * 64 * 2


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm; in one half of the draws odd, else a multiple of eight where it can be."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = n | 1 if rng.random() < 0.5 else n // 8 * 8 or n
    return max(lo, min(hi, n))


def draw(rng):
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    mode = rng.choice(("forward", "train"))
    while True:
        rows = _spread(rng, 1, 1_000_000)
        if rng.random() < 0.4:
            c = ln("", mode, rows, _spread(rng, 16, 8192), dtype, rng.choice((dtype, "fp32")))
        else:
            width = _spread(rng, 32, 2048)
            # relu's derivative jumps at 0, where the last bit of a sum decides: 32-bit gradients are compared smooth
            acts = ("silu", "gelu", "gelu_tanh") + (("relu",) if dtype != "fp32" else ())
            c = ffn("", mode, rows, width, _spread(rng, 64, 8192), dtype, rng.choice(acts), rng.random() < 0.5,
                    rng.choice((width, _spread(rng, 16, 2048))))
        del c["name"]
        # rows * hidden is bounded as well: the plain form keeps several such arrays in 32 bits
        if work(c)["flops"] <= MOST_FLOPS and rows * (c["width"] + c.get("hidden", 0)) <= 400_000_000:
            if c["op"] == "gated_ffn" or work(c)["bytes"] <= MOST_BYTES:
                return c


def work(case):
    r, d, b = case["rows"], case["width"], BYTES[case["dtype"]]
    train = case["mode"] == "train"
    if case["op"] == "layer_norm":
        p = BYTES[case["params"]] * d
        # forward: x, y, w, b; backward: x, dy and w again, dx, dw, db
        return {"bytes": 2 * r * d * b + 2 * p + (3 * r * d * b + 3 * p if train else 0),
                "flops": 8 * r * d + (12 * r * d if train else 0)}
    f, n = case["hidden"], case["out"]
    biases = (2 * f + n) * b if case["bias"] else 0
    weights = (2 * f * d + n * f) * b
    forward = r * (d + n) * b + weights + biases
    # backward: dy, x and the weights again, dx, their gradients
    backward = r * (n + 2 * d) * b + 2 * weights + biases
    flops = 4 * r * d * f + 2 * r * f * n
    return {"bytes": forward + (backward if train else 0), "flops": flops * (3 if train else 1)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    r, d = case["rows"], case["width"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    state = {"case": case}
    if case["op"] == "layer_norm":
        # residual streams drift away from zero and their rows differ in size
        scale = torch.rand(r, 1, generator=gen, device="cuda") * 3 + 0.25
        state["x"] = (torch.randn(r, d, generator=gen, device="cuda") * scale + 0.5).to(dt)
        pt = TYPES[case["params"]]
        state["w"] = normal(d, scale=0.2, shift=1.0, dtype=pt)
        state["b"] = normal(d, scale=0.2, dtype=pt)
        n = d
    else:
        f, n = case["hidden"], case["out"]
        state["x"] = normal(r, d)  # what a norm gives
        state["w_in"] = normal(2 * f, d, scale=d ** -0.5)
        state["w_out"] = normal(n, f, scale=f ** -0.5)
        state["b_in"] = normal(2 * f, scale=0.1) if case["bias"] else None
        state["b_out"] = normal(n, scale=0.1) if case["bias"] else None
    if case["mode"] == "train":
        state["dy"] = normal(r, n)
    return state


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import differentiable_sparse_iterative_gb300 as sla
    c = s["case"]
    if c["op"] == "layer_norm":
        if c["mode"] == "forward":
            return {"y": sla.sla_layernorm(s["x"], s["w"], s["b"], eps=EPS)}
        y, mean, rstd = sla.sla_layernorm(s["x"], s["w"], s["b"], eps=EPS, stats=True)
        dx, dw, db = sla.sla_layernorm_backward(s["dy"], s["x"], s["w"], mean, rstd)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    args = (s["x"], s["w_in"], s["w_out"])
    if c["mode"] == "forward":
        return {"y": sla.sla_gated_ffn(*args, s["b_in"], s["b_out"], activation=c["act"])}
    y, saved = sla.sla_gated_ffn(*args, s["b_in"], s["b_out"], activation=c["act"], save=True)
    dx, dw_in, dw_out, db_in, db_out = sla.sla_gated_ffn_backward(s["dy"], *args, saved, activation=c["act"],
                                                                  want_grad_bias=c["bias"])
    out = {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}
    if c["bias"]:
        out["db_in"], out["db_out"] = db_in, db_out
    return out


# ------------------------------------------------------------------ the plain forms, in 32 bits

def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        phi = 0.5 * (1.0 + torch.erf(g / ROOT_2))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(TANH_A * (g + TANH_B * g * g * g))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * TANH_A * (1.0 + 3.0 * TANH_B * g * g)
    return torch.clamp(g, min=0.0), (g > 0).to(g.dtype)


def _plain_ln(s, train):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    xc = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    out = {"y": (xh * w + b).to(s["x"].dtype)}
    if train:
        dy = s["dy"].float()
        dxh = dy * w
        dx = rstd * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
        out["dx"] = dx.to(s["x"].dtype)
        out["dw"] = (dy * xh).sum(0).to(s["w"].dtype)
        out["db"] = dy.sum(0).to(s["b"].dtype)
    return out


def _plain_ffn(s, train):
    c, dt = s["case"], s["x"].dtype
    f = c["hidden"]
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    gu = x @ w_in.t()
    if c["bias"]:
        gu = gu + s["b_in"].float()
    g, u = gu[:, :f], gu[:, f:]
    a, da = _act(g, c["act"])
    h = a * u
    y = h @ w_out.t()
    if c["bias"]:
        y = y + s["b_out"].float()
    out = {"y": y.to(dt)}
    if train:
        dy = s["dy"].float()
        dh = dy @ w_out
        dgu = torch.cat((dh * u * da, dh * a), 1)
        out["dx"] = (dgu @ w_in).to(dt)
        out["dw_in"] = (dgu.t() @ x).to(dt)
        out["dw_out"] = (dy.t() @ h).to(dt)
        if c["bias"]:
            out["db_in"], out["db_out"] = dgu.sum(0).to(dt), dy.sum(0).to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    plain = _plain_ln if state["case"]["op"] == "layer_norm" else _plain_ffn
    return plain(state, state["case"]["mode"] == "train")


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    """The definition in 64 bits; the gradients by differentiating it, not by the formulas above."""
    if work(case)["flops"] > MOST_FLOPS:
        return None
    s = prepare(case, seed)
    names = ("x", "w", "b") if case["op"] == "layer_norm" else ("x", "w_in", "w_out", "b_in", "b_out")
    train = case["mode"] == "train"
    v = {k: s[k].double().requires_grad_(train) for k in names if s[k] is not None}
    if case["op"] == "layer_norm":
        var, mean = torch.var_mean(v["x"], dim=1, correction=0, keepdim=True)
        y = (v["x"] - mean) * torch.rsqrt(var + EPS) * v["w"] + v["b"]
    else:
        gu = torch.nn.functional.linear(v["x"], v["w_in"], v.get("b_in"))
        g, u = gu.chunk(2, dim=1)
        act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
               "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]]
        y = torch.nn.functional.linear(act(g) * u, v["w_out"], v.get("b_out"))
    out = {"y": y.detach()}
    if train:
        grads = torch.autograd.grad(y, list(v.values()), s["dy"].double())
        out.update({"d" + k: g for k, g in zip(v, grads)})
    return out
