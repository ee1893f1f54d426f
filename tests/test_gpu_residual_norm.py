"""The residual norm on the GPU against its formulas in 64 bits (themselves checked against differentiation).

Tolerances (F = 2^-24, U the type's unit roundoff).  A result is reached by at most 60 float32 operations on values of its
size and by four sums over its row, each of at most 24 additions in sequence (16 of a thread, the rest a tree),
which move every element by at most that many F of the row's largest value: 60 + 4 * 24 < 160 F of the largest value that its
row takes on the way (`size` below), and the rounding U of the result.  A sum over the rows adds at most 160 terms in
sequence (a thread's rows, its block's warps, the blocks in strides of 32), each of which is off by 160 F: 320 F of the sum of
the terms' sizes.
"""
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
F = 2.0 ** -24
EPS = 1e-5


def randn(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def act64(g, kind):
    s = torch.sigmoid(g)
    return {"none": (g, torch.ones_like(g)), "sigmoid": (s, s * torch.sigmoid(-g)),
            "silu": (g * s, s * (1 + g * torch.sigmoid(-g)))}[kind]


def norm64(x, rms):
    xc = x if rms else x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    return xc * rstd, rstd


def back64(d, xh, rstd, rms):
    return rstd * (d - (0 if rms else d.mean(1, keepdim=True)) - xh * (d * xh).mean(1, keepdim=True))


def amax(t):
    return t.abs().amax(1, keepdim=True)


def reference(a, how, dz=None, dy=None):
    """name -> (result, its size on the way), from a dict of 64-bit tensors (or None)."""
    rms, post, kind = how["norm"] == "rms", how["post_norm"], how["gate_activation"]
    f, z, one = a["block"], a["z"], torch.ones((), dtype=torch.float64, device=DEV)
    sc, w1, w2 = (one if a[k] is None else a[k] for k in ("scale", "post_weight", "weight"))
    b1, b2 = (0 * one if a[k] is None else a[k] for k in ("post_bias", "bias"))
    fh, r1, amp1 = f, one, one
    u = f
    if post:
        fh, r1 = norm64(f, rms)
        amp1 = 1 + amax(f) * r1  # what the rounding of f's sums does to fh
        u = fh * w1 + b1
    g, dg = (one, 0 * one) if a["gate"] is None else act64(a["gate"], kind)
    t = g * u
    zn = z + sc * t
    zsize = amax(z) + amax((sc * g).abs() * ((fh.abs() + amp1) * w1.abs() + b1.abs() if post else f.abs()))
    zh, r2 = norm64(zn, rms)
    amp2 = (1 + zsize * r2) * (1 + amax(zh))
    out = {"z": (zn, zsize), "y": (zh * w2 + b2, amp2 * w2.abs().max() + b2.abs().max())}
    if dz is None and dy is None:
        return out
    D = torch.zeros_like(f) if dz is None else dz
    Dsize = amax(D)
    zero = torch.zeros_like(f)
    if dy is not None:
        D = D + back64(dy * w2, zh, r2, rms)
        Dsize = Dsize + r2 * amax(dy * w2) * (1 + amax(zh)) ** 2 * amp2
        out["weight"] = (dy * zh).sum(0), (dy.abs() * amp2).sum(0)
        out["bias"] = dy.sum(0), dy.abs().sum(0)
    usize = (amax(fh) + amp1) * w1.abs().max() + b1.abs().max() if post else amax(f)
    gsize, dgsize = (one, one) if a["gate"] is None else (amax(g) + 1, amax(dg) + 1)
    scm = sc.abs().max()
    out["dz"] = D, Dsize
    out["scale"] = (D * t).sum(0), (Dsize * gsize * usize + zero).sum(0)
    if a["gate"] is not None:
        out["dgate"] = D * sc * u * dg, Dsize * scm * usize * dgsize
    du, dusize = D * sc * g, Dsize * scm * gsize
    if post:
        out["post_weight"] = (du * fh).sum(0), (dusize * (amax(fh) + amp1) + zero).sum(0)
        out["post_bias"] = du.sum(0), (dusize + zero).sum(0)
        out["df"] = back64(du * w1, fh, r1, rms), r1 * dusize * w1.abs().max() * (1 + amax(fh)) ** 2 * amp1
    else:
        out["df"] = du, dusize
    return out


def check(got, want, what, ops):
    ref, size = want
    u = U[got.dtype]
    bound = u * ref.abs() * (1 + 2 * u) + ops * F * size + (2.0 ** -25 if got.dtype == torch.float16 else 1e-37)
    excess = (got.double() - ref).abs() - bound
    assert bool(got.isfinite().all()), what
    assert float(excess.max()) <= 0, f"{what}: {float(excess.max()):.3e} over the bound"


def tensors(rows, width, dtype, pt, seed, gate=True, post=True):
    p = {"scale": randn(width, dtype=pt, seed=seed + 3, scale=0.2, shift=0.7),
         "post_weight": randn(width, dtype=pt, seed=seed + 4, scale=0.2, shift=1.0) if post else None,
         "post_bias": randn(width, dtype=pt, seed=seed + 5, scale=0.2) if post else None,
         "weight": randn(width, dtype=pt, seed=seed + 6, scale=0.2, shift=1.0),
         "bias": randn(width, dtype=pt, seed=seed + 7, scale=0.2)}
    return {"block": randn(rows, width, dtype=dtype, seed=seed, scale=1.5, shift=0.3),
            "z": randn(rows, width, dtype=dtype, seed=seed + 1, scale=2.0, shift=0.5),
            "gate": randn(rows, width, dtype=dtype, seed=seed + 2) if gate else None, **p}


def double(a):
    return {k: None if v is None else v.double() for k, v in a.items()}


ROWS = ("dz", "df", "dgate")


def check_grads(g, want):
    named = {"df": g.block, "dz": g.z, "dgate": g.gate, "scale": g.scale, "post_weight": g.post_weight,
             "post_bias": g.post_bias, "weight": g.weight, "bias": g.bias}
    for k, t in named.items():
        assert (t is None) == (k not in want), k
        if t is not None:
            check(t, want[k], k, 160 if k in ROWS else 320)


SHAPES = [(1, 1), (3, 2), (5, 7), (1, 64), (33, 64), (257, 96), (64, 250), (2, 1001), (19, 1024), (5003, 136), (300, 256),
          (7, 4099), (9, 4096), (3, 4104), (5, 8192), (4, 8191), (3, 8183), (3, 8200), (2, 20001), (70000, 8), (50, 3), (90, 9)]
HOWS = [dict(norm="layer", post_norm=True, gate_activation="sigmoid"), dict(norm="rms", post_norm=True, gate_activation="silu"),
        dict(norm="layer", post_norm=False, gate_activation="none"), dict(norm="rms", post_norm=True, gate_activation="")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", SHAPES)
def test_forward_and_backward(rows, width, dtype):
    dz, dy = randn(rows, width, dtype=dtype, seed=50), randn(rows, width, dtype=dtype, seed=51)
    for i, how in enumerate(HOWS):
        pt = torch.float32 if i % 2 else dtype
        how = dict(how)
        gate = how["gate_activation"] != ""
        how["gate_activation"] = how["gate_activation"] or "none"
        a = tensors(rows, width, dtype, pt, 10 + i, gate, how["post_norm"])
        want = reference(double(a), how, dz.double(), dy.double())
        z, y, stats = sla.sla_residual_norm(**a, **how, stats=True)
        check(z, want.pop("z"), "z", 160)
        check(y, want.pop("y"), "y", 160)
        again = sla.sla_residual_norm(**a, **how)
        assert torch.equal(z, again[0]) and torch.equal(y, again[1])
        given = {k: v for k, v in a.items() if k not in ("bias", "block", "z")}
        args = (a["block"], a["z"], stats)
        g = sla.sla_residual_norm_backward(dz, dy, *args, **given, **how)
        check_grads(g, want)
        g2 = sla.sla_residual_norm_backward(dz, dy, *args, **given, **how)
        assert all(p is q or torch.equal(p, q) for p, q in zip(g, g2))
        if i == 0:
            for up in ((dz, None), (None, dy)):
                part = sla.sla_residual_norm_backward(*up, *args, **given, **how)
                want = reference(double(a), how, *(None if t is None else t.double() for t in up))
                check_grads(part, {k: v for k, v in want.items() if k not in ("z", "y")})
            alone = sla.sla_residual_norm_backward(dz, dy, *args, **given, **how, want_grad_params=False)
            assert torch.equal(alone.block, g.block) and alone.scale is None
            only, none = sla.sla_residual_norm(**a, **how, next_norm=False)
            assert none is None and torch.equal(only, z)


def test_the_formulas_are_those_of_differentiation():
    for i, how in enumerate(HOWS):
        how = dict(how, gate_activation=how["gate_activation"] or "none")
        a = double(tensors(7, 12, torch.float32, torch.float32, 60 + i, how["gate_activation"] != "none", how["post_norm"]))
        leaves = {k: v.requires_grad_() for k, v in a.items() if v is not None}
        out = reference(a, how)
        dz, dy = randn(7, 12, dtype=torch.float64, seed=70), randn(7, 12, dtype=torch.float64, seed=71)
        got = torch.autograd.grad([out["z"][0], out["y"][0]], list(leaves.values()), [dz, dy])
        want = reference({k: None if v is None else v.detach() for k, v in a.items()}, how, dz, dy)
        name = {"block": "df", "z": "dz", "gate": "dgate"}
        for k, g in zip(leaves, got):
            assert float((g - want[name.get(k, k)][0]).abs().max()) < 1e-11, k


def test_absent_parameters_are_ones_and_zeros():
    rows, width = 40, 72
    for dtype in TYPES:
        a = tensors(rows, width, dtype, dtype, 80)
        bare = {k: a[k] for k in ("block", "z")}
        how = dict(norm="layer", post_norm=True, gate_activation="none")
        full = dict.fromkeys(("gate", "scale", "post_weight", "post_bias", "weight", "bias"))
        want = reference(double({**full, **bare}), how, a["gate"].double(), a["gate"].double())
        z, y, stats = sla.sla_residual_norm(**bare, stats=True)
        check(z, want.pop("z"), "z", 160)
        check(y, want.pop("y"), "y", 160)
        for pt in (dtype, torch.float32):
            g = sla.sla_residual_norm_backward(a["gate"], a["gate"], *bare.values(), stats, param_dtype=pt)
            check_grads(g, want)
            assert g.scale.dtype == pt and g.weight.dtype == pt


def test_autograd_and_differences():
    rows, width = 21, 70
    a = tensors(rows, width, torch.float32, torch.float32, 90)
    how = dict(norm="layer", gate_activation="silu")
    leaves = {k: v.clone().requires_grad_() for k, v in a.items()}
    dz, dy = randn(rows, width, dtype=torch.float32, seed=98), randn(rows, width, dtype=torch.float32, seed=99)
    torch.autograd.backward(sla.residual_norm(**leaves, **how), [dz, dy])

    def loss(b):
        z, y = sla.residual_norm(**b, **how)
        return float((z.double() * dz).sum() + (y.double() * dy).sum())

    for i, (k, t) in enumerate(leaves.items()):
        v, step = randn(*t.shape, dtype=torch.float32, seed=100 + i), 1e-2
        with torch.no_grad():
            f = [loss({**a, k: a[k] + sign * step * v}) for sign in (1, -1)]
        d = (f[0] - f[1]) / (2 * step)
        # step^2 / 6 times the third derivative, of order one a term, and float32 roundings over the step
        size = float((t.grad.double() * v.double()).abs().sum())
        assert abs(d - float((t.grad.double() * v.double()).sum())) <= 3e-3 * size, k
    # one result, some leaves
    z, y = sla.residual_norm(leaves["block"], a["z"], weight=leaves["weight"], norm="rms")
    got = torch.autograd.grad(y, [leaves["block"], leaves["weight"]], dy)
    assert all(g.isfinite().all() for g in got)
    z, y = sla.residual_norm(leaves["block"], a["z"], next_norm=False)
    assert y is None and torch.autograd.grad(z, leaves["block"], dz)[0].shape == z.shape


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [64, 63, 9000])
def test_layouts(width, dtype):
    rows = 33
    how = dict(norm="layer", post_norm=True, gate_activation="sigmoid")
    a = tensors(rows, width, dtype, dtype, 110)
    z, y = sla.sla_residual_norm(**a, **how)
    wide = torch.cat([a["block"], a["z"], a["gate"], a["gate"][:, :3]], -1)
    views = dict(a, block=wide[:, :width], z=wide[:, width:2 * width], gate=wide[:, 2 * width:3 * width])
    # (other vectors, other orders of a row's sums)
    want = reference(double(a), how)
    z2, y2 = sla.sla_residual_norm(**views, **how)
    check(z2, want["z"], "z", 160)
    check(y2, want["y"], "y", 160)
    three = {k: (v.view(3, 11, width) if k in ("block", "z", "gate") else v) for k, v in a.items()}
    z3, y3 = sla.residual_norm(**three, **how)
    assert torch.equal(z3.view(rows, width), z) and torch.equal(y3.view(rows, width), y)
    turned = dict(a, block=a["block"].t().contiguous().t())
    assert torch.equal(sla.residual_norm(**turned, **how)[1], y)
    odd = {}
    for k in ("scale", "post_weight", "post_bias", "weight", "bias"):  # parameters of no alignment
        odd[k] = torch.empty(width + 1, dtype=dtype, device=DEV)[1:].copy_(a[k])
    z4, y4 = sla.sla_residual_norm(**{**a, **odd}, **how)
    assert torch.equal(z4, z) and torch.equal(y4, y)


@pytest.mark.parametrize("width", [64, 63, 9000])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_no_number_stays_in_its_row(width, value):
    rows = 37
    a = tensors(rows, width, torch.bfloat16, torch.float32, 120)
    how = dict(norm="layer", post_norm=True, gate_activation="sigmoid")
    z, y, stats = sla.sla_residual_norm(**a, **how, stats=True)
    for k in ("block", "z"):
        b = dict(a, **{k: a[k].clone()})
        b[k][5, 3] = value
        z2, y2, stats2 = sla.sla_residual_norm(**b, **how, stats=True)
        others = [r for r in range(rows) if r != 5]
        assert torch.equal(z2[others], z[others]) and torch.equal(y2[others], y[others])
        assert not bool(y2[5].isfinite().any())
        given = {q: b[q] for q in ("gate", "scale", "post_weight", "post_bias", "weight")}
        g = sla.sla_residual_norm_backward(z, y, b["block"], b["z"], stats2, **given, **how)
        assert bool(g.block[others].isfinite().all()) and bool(g.z[others].isfinite().all())
    # rows that are constant, or large: nothing but what the formula says
    flat = dict(a, block=torch.full_like(a["block"], 3e4), z=torch.full_like(a["z"], -2e4))
    for norm in ("layer", "rms"):
        h = dict(how, norm=norm)
        z3, y3, s3 = sla.sla_residual_norm(**flat, **h, stats=True)
        given = {q: flat[q] for q in ("gate", "scale", "post_weight", "post_bias", "weight")}
        g = sla.sla_residual_norm_backward(z, y, flat["block"], flat["z"], s3, **given, **h)
        assert all(bool(t.isfinite().all()) for t in (z3, y3, *g))


def test_no_rows():
    x = torch.empty(0, 24, dtype=torch.float16, device=DEV)
    z, y, stats = sla.sla_residual_norm(x, x, stats=True)
    assert z.shape == y.shape == x.shape
    g = sla.sla_residual_norm_backward(x, x, x, x, stats)
    assert g.scale.shape == (24,) and not any(bool(t.any()) for t in g[3:])


def test_streams_and_graphs():
    a = tensors(3000, 200, torch.bfloat16, torch.bfloat16, 130)
    how = dict(norm="rms", post_norm=True, gate_activation="silu")
    given = {q: a[q] for q in ("gate", "scale", "post_weight", "post_bias", "weight")}
    dz = randn(3000, 200, dtype=torch.bfloat16, seed=140)

    def call(ws=None):
        z, y, stats = sla.sla_residual_norm(**a, **how, stats=True)
        return (z, y, *sla.sla_residual_norm_backward(dz, dz, a["block"], a["z"], stats, **given, **how, workspace=ws))

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(ws)
        graphs.append((graph, out))
    for _ in range(2):
        for graph, out in graphs:
            out[2].zero_()
            graph.replay()
            assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_refusals():
    x = randn(6, 16, dtype=torch.float16, seed=150)
    w = torch.ones(16, dtype=torch.float16, device=DEV)
    z, y, stats = sla.sla_residual_norm(x, x, weight=w, stats=True)
    for call, message in (
            (lambda: sla.sla_residual_norm(x, x[:3]), "z must have"),
            (lambda: sla.sla_residual_norm(x, x, x.float()), "gate must have"),
            (lambda: sla.sla_residual_norm(x.double(), x.double()), "float32, float16"),
            (lambda: sla.sla_residual_norm(x.t(), x.t()), "contiguous"),
            (lambda: sla.sla_residual_norm(x, x, scale=w[:4]), "scale must have"),
            (lambda: sla.sla_residual_norm(x, x, weight=w.bfloat16()), "parameters must have"),
            (lambda: sla.sla_residual_norm(x, x, weight=w, bias=w.float()), "bias must have"),
            (lambda: sla.sla_residual_norm(x, x, norm="batch"), "unknown norm"),
            (lambda: sla.sla_residual_norm(x, x, gate_activation="relu"), "unknown gate activation"),
            (lambda: sla.sla_residual_norm_backward(x[:2], x, x, x, stats, weight=w), "dz must have"),
            (lambda: sla.sla_residual_norm_backward(x, x[:2], x, x, stats, weight=w), "dy must have"),
            (lambda: sla.sla_residual_norm_backward(x, x, x, x, stats[:2], weight=w), "stats must have"),
            (lambda: sla.sla_residual_norm_backward(x, x, x, x, stats, param_dtype=torch.float64), "param_dtype"),
            (lambda: sla.sla_residual_norm(x, x.cpu()), "CUDA tensor")):
        with pytest.raises(ValueError, match=message):
            call()
    for eps in (-1.0, float("nan")):
        with pytest.raises(sla.SlaError):
            sla.sla_residual_norm(x, x, eps=eps)
