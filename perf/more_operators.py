"""What is measured of the linear layer, the residual norm and the gated scan.

With the layer norm and the gated feed-forward block they make a network that predicts a matrix's coefficients from
features of the grid cells, one token a cell (a 64 x 64 grid has 4,096, a 1000 x 1000 grid 1,000,000): a linear layer
makes the scan's inputs and gates, the scan carries information along the lines of the grid (or along one path
through all cells), a linear layer leads back, and the residual norm joins a block's result with the residual stream.
A case is one forward call ("forward": inference) or a training step's forward and backward call ("train").

    linear         y = act(x W^T + b) + r,  W [out, width]
    residual norm  z' = z + scale * act(gate) * N(f; w1, b1),  y = N(z'; w2, b2)
                   N(x; w, b) = (x - mean x) / sqrt(var x + eps) * w + b ("layer"), or without the mean ("rms")
    gated scan     h_t = a_t h_{t-1} + (1 - a_t) x_t,  a = 1 / (1 + e^-gate), along each sequence, from its state
"""
import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
TANH_A, TANH_B = math.sqrt(2.0 / math.pi), 0.044715


def linear(name, mode, rows, width, out, dtype, act="none", bias=True, residual=False):
    return {"name": name, "op": "linear", "mode": mode, "rows": rows, "width": width, "out": out, "dtype": dtype,
            "act": act, "bias": bias, "residual": residual}


def norm(name, mode, rows, width, dtype, kind="layer", gate="none", params=None, post=True):
    """gate: an activation, or "" for no gate; post: f is normed before it is added."""
    return {"name": name, "op": "residual_norm", "mode": mode, "rows": rows, "width": width, "dtype": dtype,
            "kind": kind, "gate": gate, "params": params or dtype, "post": post}


def scan(name, mode, sequences, tokens, channels, dtype, ragged=False, reverse=False):
    """tokens: of all sequences together; ragged: of random lengths, some of them empty, with rows behind the last."""
    return {"name": name, "op": "gated_scan", "mode": mode, "sequences": sequences, "tokens": tokens,
            "channels": channels, "dtype": dtype, "ragged": ragged, "reverse": reverse}


def listed():
    return [
        # one query point through a trained network's wide layer: the weights are read once and little else
        linear("linear one token", "forward", 1, 1024, 4096, "bf16", "silu"),
        # the layer back to the residual stream on every cell of a 1000 x 1000 grid
        linear("linear 1000x1000", "forward", 1_000_000, 64, 64, "bf16", residual=True),
        # training on a 64 x 64 grid in the solver's single precision
        linear("linear 64x64 fp32 train", "train", 4096, 256, 512, "fp32", "gelu"),
        # sizes that divide nothing
        linear("linear odd train", "train", 2049, 250, 131, "fp16", "relu", residual=True),
        # training a wide network on a batch of two 128 x 128 grids: inputs and gates of a scan in one
        linear("linear 2x128x128 wide train", "train", 32768, 1024, 2048, "bf16"),
        # one query point: latency
        norm("norm one row", "forward", 1, 1024, "bf16", gate="sigmoid"),
        # every cell of the 1000 x 1000 grid
        norm("norm 1000x1000 train", "train", 1_000_000, 64, "bf16", gate="sigmoid"),
        # odd sizes, parameters kept in 32 bits
        norm("norm odd train", "train", 5003, 1001, "fp16", kind="rms", gate="silu", params="fp32"),
        # one step of 64 sequences that are continued token by token
        scan("scan 64 single tokens", "forward", 64, 64, 1024, "bf16"),
        # the lines of a 1000 x 1000 grid
        scan("scan 1000 lines train", "train", 1000, 1_000_000, 64, "bf16"),
        # one path through all cells of that grid, in single precision
        scan("scan one path", "forward", 1, 1_000_000, 64, "fp32"),
        # boundary curves of 57 objects, of different lengths, packed one behind another, walked backwards
        scan("scan ragged train", "train", 57, 60_001, 333, "fp16", ragged=True, reverse=True),
    ]


MOST_FLOPS = 6 * 32768 * 1024 * 2048  # the largest listed cases'
MOST_ELEMENTS = 64_000_000


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm; in one half of the draws odd, else a multiple of eight where it can be."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = n | 1 if rng.random() < 0.5 else n // 8 * 8 or n
    return max(lo, min(hi, n))


def draw(rng):
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    mode = rng.choice(("forward", "train"))
    op = rng.choice(("linear", "residual_norm", "gated_scan"))
    while True:
        rows = _spread(rng, 1, 1_000_000)
        if op == "linear":
            # relu's derivative jumps at 0, where the last bit of a sum decides: 32-bit gradients are compared smooth
            acts = ("none", "silu", "gelu", "gelu_tanh") + (("relu",) if dtype != "fp32" else ())
            c = linear("", mode, rows, _spread(rng, 16, 4096), _spread(rng, 1, 4096), dtype, rng.choice(acts),
                       rng.random() < 0.7, rng.random() < 0.5)
            fits = work(c)["flops"] <= MOST_FLOPS and rows * (c["width"] + c["out"]) <= 200_000_000
        elif op == "residual_norm":
            c = norm("", mode, rows, _spread(rng, 16, 8192), dtype, rng.choice(("layer", "rms")),
                     rng.choice(("", "none", "sigmoid", "silu")), rng.choice((dtype, "fp32")), rng.random() < 0.7)
            fits = rows * c["width"] <= MOST_ELEMENTS
        else:
            n = _spread(rng, 1, rows)
            ragged = rng.random() < 0.5
            c = scan("", mode, n, rows if ragged else max(1, rows // n) * n, _spread(rng, 8, 4096), dtype, ragged,
                     rng.random() < 0.5)
            fits = c["tokens"] * c["channels"] <= MOST_ELEMENTS
        if fits:
            del c["name"]
            return c


def work(case):
    b, train = BYTES[case["dtype"]], case["mode"] == "train"
    if case["op"] == "linear":
        r, d, n = case["rows"], case["width"], case["out"]
        bias = n * b if case["bias"] else 0
        forward = (r * (d + n) + n * d) * b + bias + (r * n * b if case["residual"] else 0)
        backward = (r * (n + 2 * d) + 2 * n * d) * b + bias  # dy, x and W again, dx, dW, db
        return {"bytes": forward + (backward if train else 0), "flops": 2 * r * d * n * (3 if train else 1)}
    if case["op"] == "residual_norm":
        r, d = case["rows"], case["width"]
        gate = 1 if case["gate"] else 0
        params = (5 if case["post"] else 3) * d * BYTES[case["params"]]
        # f, z, gate, z', y; backward: f, z, gate, dz', dy, df, dz, dgate
        return {"bytes": ((4 + gate) + ((6 + 2 * gate) if train else 0)) * r * d * b + params * (3 if train else 1),
                "flops": (20 + (50 if train else 0)) * r * d}
    n, c = case["tokens"], case["channels"]
    states = 4 * case["sequences"] * c
    # x, gate, h and the states; backward: dh, x, gate, dx, dgate and the states' gradients
    return {"bytes": (3 + (5 if train else 0)) * n * c * b + states * (5 if train else 2),
            "flops": (8 + (24 if train else 0)) * n * c}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    s = {"case": case}
    train = case["mode"] == "train"
    if case["op"] == "linear":
        r, d, n = case["rows"], case["width"], case["out"]
        s["x"] = normal(r, d)  # what a norm gives
        s["w"] = normal(n, d, scale=d ** -0.5)
        s["b"] = normal(n, scale=0.1) if case["bias"] else None
        s["r"] = normal(r, n) if case["residual"] else None
        if train:
            s["dy"] = normal(r, n)
    elif case["op"] == "residual_norm":
        r, d = case["rows"], case["width"]
        pt = TYPES[case["params"]]
        # a block's results and residual streams drift away from zero and their rows differ in size
        size = torch.rand(r, 1, generator=gen, device="cuda") * 3 + 0.25
        s["f"] = (torch.randn(r, d, generator=gen, device="cuda") * size + 0.3).to(dt)
        s["z"] = (torch.randn(r, d, generator=gen, device="cuda") * size + 0.5).to(dt)
        s["gate"] = normal(r, d) if case["gate"] else None
        s["scale"] = normal(d, scale=0.2, shift=0.7, dtype=pt)
        s["w1"] = normal(d, scale=0.2, shift=1.0, dtype=pt) if case["post"] else None
        s["b1"] = normal(d, scale=0.2, dtype=pt) if case["post"] else None
        s["w2"] = normal(d, scale=0.2, shift=1.0, dtype=pt)
        s["b2"] = normal(d, scale=0.2, dtype=pt)
        if train:
            s["dz"], s["dy"] = normal(r, d), normal(r, d)
    else:
        q, n, c = case["sequences"], case["tokens"], case["channels"]
        # inputs and gates are the halves of a linear layer's rows; most gates are open, so that states last
        both = torch.empty(n, 2 * c, dtype=dt, device="cuda")
        both[:, :c] = normal(n, c)
        both[:, c:] = normal(n, c, scale=1.5, shift=2.0)
        s["state"] = normal(q, c, dtype=torch.float32)
        s["offsets"], s["starts"], s["end"], s["most"] = None, None, n, max(1, n // q)
        if case["ragged"]:
            rng = random.Random(seed)
            end = n - rng.randrange(0, n // 8 + 1)  # rows behind the last sequence
            cuts = sorted(rng.randrange(0, end + 1) for _ in range(q - 1))
            marks = [0] + cuts + [end]
            s["end"], s["most"] = end, max(1, max(b - a for a, b in zip(marks, marks[1:])))
            s["offsets"] = torch.tensor(marks, dtype=torch.int32, device="cuda")
        else:
            both = both.view(q, n // q, 2 * c)
        s["x"], s["g"] = both[..., :c], both[..., c:]
        if train:
            s["dh"] = normal(n, c).view(s["x"].shape)
            s["dfinal"] = normal(q, c, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import differentiable_sparse_iterative_gb300 as sla
    c = s["case"]
    train = c["mode"] == "train"
    if c["op"] == "linear":
        args = (s["x"], s["w"], s["b"])
        if not train:
            return {"y": sla.sla_linear(*args, residual=s["r"], activation=c["act"])}
        y, saved = sla.sla_linear(*args, residual=s["r"], activation=c["act"], save=True)
        dx, dw, db = sla.sla_linear_backward(s["dy"], s["x"], s["w"], saved, activation=c["act"],
                                             want_grad_bias=c["bias"])
        out = {"y": y, "dx": dx, "dw": dw}
        if c["bias"]:
            out["db"] = db
        return out
    if c["op"] == "residual_norm":
        how = {"norm": c["kind"], "post_norm": c["post"], "gate_activation": c["gate"] or "none", "eps": EPS}
        params = {"gate": s["gate"], "scale": s["scale"], "post_weight": s["w1"], "post_bias": s["b1"]}
        if not train:
            z, y = sla.sla_residual_norm(s["f"], s["z"], weight=s["w2"], bias=s["b2"], **params, **how)
            return {"z": z, "y": y}
        z, y, stats = sla.sla_residual_norm(s["f"], s["z"], weight=s["w2"], bias=s["b2"], **params, **how, stats=True)
        g = sla.sla_residual_norm_backward(s["dz"], s["dy"], s["f"], s["z"], stats, weight=s["w2"], **params, **how)
        out = {"z": z, "y": y, "df": g.block, "dz": g.z, "dscale": g.scale, "dw2": g.weight, "db2": g.bias}
        if s["gate"] is not None:
            out["dgate"] = g.gate
        if c["post"]:
            out["dw1"], out["db1"] = g.post_weight, g.post_bias
        return out
    how = {"state": s["state"], "offsets": s["offsets"], "reverse": c["reverse"]}
    if not train:
        h, final = sla.sla_gated_scan(s["x"], s["g"], **how)
        return {"h": h, "final": final}
    h, final, saved = sla.sla_gated_scan(s["x"], s["g"], **how, save=True)
    dx, dg, dstate = sla.sla_gated_scan_backward(s["dh"], s["x"], s["g"], saved, dfinal=s["dfinal"], **how)
    return {"h": h, "final": final, "dx": dx, "dgate": dg, "dstate": dstate}


# ------------------------------------------------------------------ the plain forms, in 32 bits

def _sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g))


def _act(p, kind):
    """act(p) and act'(p)."""
    if kind == "none":
        return p, torch.ones_like(p)
    if kind == "sigmoid":
        s = _sigmoid(p)
        return s, s * _sigmoid(-p)
    if kind == "silu":
        s = _sigmoid(p)
        return p * s, s * (1.0 + p * (1.0 - s))
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-p / math.sqrt(2.0))
        return p * phi, phi + p * torch.exp(-0.5 * p * p) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        s = _sigmoid(2.0 * TANH_A * (p + TANH_B * p * p * p))
        return p * s, s + 2.0 * p * s * (1.0 - s) * TANH_A * (1.0 + 3.0 * TANH_B * p * p)
    return torch.clamp(p, min=0.0), (p > 0).to(p.dtype)


def _plain_linear(s, train):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    p = x @ w.t()
    if c["bias"]:
        p = p + s["b"].float()
    a, da = _act(p, c["act"])
    out = {"y": (a + s["r"].float() if c["residual"] else a).to(dt)}
    if train:
        dp = s["dy"].float() * da
        out["dx"], out["dw"] = (dp @ w).to(dt), (dp.t() @ x).to(dt)
        if c["bias"]:
            out["db"] = dp.sum(0).to(dt)
    return out


def _normed(x, kind):
    """The rows without their mean, over their deviation; and one over that."""
    xc = x - x.mean(1, keepdim=True) if kind == "layer" else x
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    return xc * rstd, rstd


def _normed_back(d, xh, rstd, kind):
    d = d - xh * (d * xh).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if kind == "layer" else 0.0)
    return d * rstd


def _plain_norm(s, train):
    c, dt, pt = s["case"], s["f"].dtype, s["w2"].dtype
    f, z, scale, w2, b2 = (s[k].float() for k in ("f", "z", "scale", "w2", "b2"))
    u = f
    if c["post"]:
        w1, b1 = s["w1"].float(), s["b1"].float()
        fh, frstd = _normed(f, c["kind"])
        u = fh * w1 + b1
    a = None
    if c["gate"]:
        a, da = _act(s["gate"].float(), c["gate"])
    au = u if a is None else a * u
    znew = z + scale * au
    zh, zrstd = _normed(znew, c["kind"])
    out = {"z": znew.to(dt), "y": (zh * w2 + b2).to(dt)}
    if not train:
        return out
    dy = s["dy"].float()
    out["dw2"], out["db2"] = (dy * zh).sum(0).to(pt), dy.sum(0).to(pt)
    dz = s["dz"].float() + _normed_back(dy * w2, zh, zrstd, c["kind"])
    out["dz"] = dz.to(dt)
    out["dscale"] = (dz * au).sum(0).to(pt)
    du = dz * scale
    if a is not None:
        out["dgate"] = (du * u * da).to(dt)
        du = du * a
    if c["post"]:
        out["dw1"], out["db1"] = (du * fh).sum(0).to(pt), du.sum(0).to(pt)
        du = _normed_back(du * w1, fh, frstd, c["kind"])
    out["df"] = du.to(dt)
    return out


def _recur(a, v, most):
    """v_t + a_t v_{t-1} + a_t a_{t-1} v_{t-2} + ...: spans of rows are joined, twice as long each time, up to `most`."""
    d = 1
    while d < most:
        v = torch.cat((v[:d], v[d:] + a[d:] * v[:-d]))
        if 2 * d < most:
            a = torch.cat((a[:d], a[d:] * a[:-d]))
        d *= 2
    return v


def _bounds(s):
    """Each sequence's first row and the row behind its last."""
    if s["offsets"] is not None:
        return s["offsets"][:-1].long(), s["offsets"][1:].long()
    q, n = s["case"]["sequences"], s["case"]["tokens"]
    first = torch.arange(q, device="cuda") * (n // q)
    return first, first + n // q


def _plain_scan(s, train):
    c, dt = s["case"], s["x"].dtype
    n, end, shape = c["channels"], s["end"], s["x"].shape
    x, g = s["x"].reshape(-1, n)[:end].float(), s["g"].reshape(-1, n)[:end].float()
    begin, stop = _bounds(s)
    some = stop > begin
    begin, last = begin[some], stop[some] - 1
    if c["reverse"]:  # the sequences mirrored, and so their order of rows
        x, g, begin, last = x.flip(0), g.flip(0), end - 1 - last, end - 1 - begin
    state = s["state"][some]
    a, b = _sigmoid(g), _sigmoid(-g)

    def rows(t):
        t = t.flip(0) if c["reverse"] else t
        return torch.cat((t, t.new_zeros(c["tokens"] - end, n))).to(dt).view(shape)

    v = b * x
    v[begin] += a[begin] * state
    inner = a.clone()
    inner[begin] = 0.0
    h = _recur(inner, v, s["most"])
    final = s["state"].clone()
    final[some] = h[last]
    out = {"h": rows(h), "final": final}
    if train:
        dh = s["dh"].reshape(-1, n)[:end].float()
        dh = dh.flip(0).clone() if c["reverse"] else dh.clone()
        dh[last] += s["dfinal"][some]
        # l_t = dh_t + a_{t+1} l_{t+1}, the gradient of h_t
        after = torch.cat((inner[1:], inner.new_zeros(min(1, end), n)))
        l = _recur(after.flip(0), dh.flip(0), s["most"]).flip(0)
        before = torch.cat((h.new_zeros(min(1, end), n), h[:-1]))
        before[begin] = state
        out["dx"], out["dgate"] = rows(l * b), rows(l * (before - x) * a * b)
        dstate = s["dfinal"].clone()
        dstate[some] = a[begin] * l[begin]
        out["dstate"] = dstate
    return out


def run(state):
    if own:
        return _run_own(state)
    plain = {"linear": _plain_linear, "residual_norm": _plain_norm, "gated_scan": _plain_scan}[state["case"]["op"]]
    return plain(state, state["case"]["mode"] == "train")


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_linear(s, v):
    c = s["case"]
    y = torch.nn.functional.linear(v["x"], v["w"], v.get("b"))
    y = {"none": lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[c["act"]](y)
    return {"y": y + s["r"].double() if c["residual"] else y}


def _exact_norm(s, v):
    c = s["case"]

    def normed(x, w, b):
        if c["kind"] == "layer":
            return torch.nn.functional.layer_norm(x, x.shape[1:], w, b, EPS)
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w + b

    u = normed(v["f"], v["w1"], v["b1"]) if c["post"] else v["f"]
    if c["gate"]:
        u = u * {"none": lambda t: t, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[c["gate"]](v["gate"])
    z = torch.addcmul(v["z"], v["scale"], u)
    return {"z": z, "y": normed(z, v["w2"], v["b2"])}


def _exact_scan(s, v):
    """Row after row within blocks of about sqrt(rows) rows, all blocks side by side, then block after block."""
    c, end = s["case"], s["end"]
    n = c["channels"]
    x, g = v["x"].reshape(-1, n)[:end], v["g"].reshape(-1, n)[:end]
    begin, stop = (t.tolist() for t in _bounds(s))
    pairs = [(i, p, q - 1) for i, (p, q) in enumerate(zip(begin, stop)) if q > p]
    if c["reverse"]:
        x, g = x.flip(0), g.flip(0)
        pairs = [(i, end - 1 - q, end - 1 - p) for i, p, q in pairs]
    some = torch.tensor([p[0] for p in pairs], device="cuda")
    first = torch.tensor([p[1] for p in pairs], device="cuda")
    last = torch.tensor([p[2] for p in pairs], device="cuda")
    final = v["state"]
    if not pairs:
        return {"h": v["x"] * 0.0, "final": final}
    a = torch.sigmoid(g)
    into = torch.zeros_like(x).index_copy(0, first, a[first] * v["state"][some])
    u = torch.sigmoid(-g) * x + into
    a = a * torch.ones(end, 1, dtype=a.dtype, device="cuda").index_fill(0, first, 0.0)
    size = max(1, math.isqrt(end))
    blocks = -(-end // size)
    pad = (0, 0, 0, blocks * size - end)
    a = torch.nn.functional.pad(a, pad).view(blocks, size, n).unbind(1)
    u = torch.nn.functional.pad(u, pad).view(blocks, size, n).unbind(1)
    h, p, hs, ps = u[0], a[0], [u[0]], [a[0]]
    for k in range(1, size):
        h, p = torch.addcmul(u[k], a[k], h), a[k] * p
        hs.append(h)
        ps.append(p)
    carry, into = torch.zeros_like(h[0]), []
    for hb, pb in zip(h.unbind(0), p.unbind(0)):
        into.append(carry)
        carry = torch.addcmul(hb, pb, carry)
    h = torch.stack(hs, 1) + torch.stack(ps, 1) * torch.stack(into)[:, None]
    h = h.reshape(blocks * size, n)[:end]
    final = final.index_copy(0, some, h[last])
    h = h.flip(0) if c["reverse"] else h
    return {"h": torch.nn.functional.pad(h, (0, 0, 0, c["tokens"] - end)).view(v["x"].shape), "final": final}


def exact(case, seed):
    """The definition in 64 bits; the gradients by differentiating it, not by the formulas above."""
    if case["op"] == "linear" and work(case)["flops"] > MOST_FLOPS:
        return None
    s = prepare(case, seed)
    train = case["mode"] == "train"
    names, of, grads = {
        "linear": (("x", "w", "b"), _exact_linear, {"y": "dy"}),
        "residual_norm": (("f", "z", "gate", "scale", "w1", "b1", "w2", "b2"), _exact_norm, {"z": "dz", "y": "dy"}),
        "gated_scan": (("x", "g", "state"), _exact_scan, {"h": "dh", "final": "dfinal"}),
    }[case["op"]]
    v = {k: s[k].double().requires_grad_(train) for k in names if s[k] is not None}
    out = of(s, v)
    if train:
        wanted = [(out[k], s[g].double()) for k, g in grads.items() if out[k].requires_grad]
        got = torch.autograd.grad([o for o, _ in wanted], list(v.values()), [g for _, g in wanted])
        called = {"g": "dgate"}
        out.update({called.get(k, "d" + k): g for k, g in zip(v, got)})
    return {k: t.detach() for k, t in out.items()}
