"""The gated scan where gates keep a state over many rows: 1 - a is small there, and what it lets in is most of h when the state is.

Errors are relative to the results themselves, channel by channel (each has a mean gate of its own), in L2, against the
definition in 64 bits.  F = 2^-24:
    1 - a     2^-22 of the exponential and 2^-23 of the reciprocal by approximation, their sum's and product's roundings: 2^-20;
              with 16-bit data the exponent's rounding too, |g| 2^-23
    a step    rounds h once, by F of it, and what it adds to h three times: n F after n rows at most, or, where their signs
              are random (inputs are, and no state outweighs them), sqrt(n) F, allowed four times
    a map of a tile, joined with others: eight roundings more
A row's errors are relative to the two parts that it adds, a |h| and (1 - a) |x| (|dh| and a |l| backward), whatever becomes of their sum: the
state behind the last row, one value a sequence that may have come out small, is measured against the root mean square of its
channel's parts along the rows where that is more.
"""
import numpy as np
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half of the smallest number's distance to zero
F = 2.0 ** -24
GATES = [4, 5, 6, 8, 10, 11, 12, 13, 14, 15, 16, 17, 18, 24, 30, -2, -8]

#            sequences, rows, channels
SHAPES = [(5, 1, 64),      # single steps
          (3, 40, 33),     # one tile, channels one by one
          (1, 100, 64), (7, 1000, 66), (2, 900, 35),  # tiles that look back
          (1, 20_000, 34),
          (760, 100, 34), (800, 300, 17 * 2)]  # a warp walks along each


def f64(t):
    return t.detach().double().cpu().numpy()


def scan64(x, g, s, reverse=False):
    """h, all states before a row, the last, and the parts of h, of [sequences, rows, channels]."""
    a, b = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    h, before = np.zeros_like(x), np.zeros_like(x)
    rows = range(x.shape[1])
    for t in reversed(rows) if reverse else rows:
        before[:, t] = s
        s = a[:, t] * s + b[:, t] * x[:, t]
        h[:, t] = s
    return h, before, s, a * np.abs(before) + b * np.abs(x)


def back64(x, g, before, dh, m, reverse=False):
    a, b = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    l = np.zeros_like(x)
    rows = range(x.shape[1])
    for t in rows if reverse else reversed(rows):
        l[:, t] = dh[:, t] + m
        m = a[:, t] * l[:, t]
    return b * l, l * (before - x) * a * b, m, np.abs(dh) + a * np.abs(l)


def data(shape, dtype, spread, constant, state, seed=1):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    mean = torch.tensor([GATES[i % len(GATES)] for i in range(shape[2])], device=DEV)
    x = torch.ones(shape, device=DEV, dtype=dtype) if constant else randn(*shape).to(dtype)
    g = (mean + spread * randn(*shape)).to(dtype)
    return x, g, randn(shape[0], shape[2]) if state else None


def check(got, want, g, rows, dtype, systematic, what, along=None):
    """Channel by channel, relative to the channel (or to the root mean square of `along`, [sequences, rows, channels])."""
    got = f64(got).reshape(want.shape)
    over = tuple(range(want.ndim - 1))
    size = np.sqrt((want ** 2).sum(over))
    if along is not None:
        size = np.maximum(size, np.sqrt((along ** 2).mean(1).sum(0)))
    err = np.sqrt(((got - want) ** 2).sum(over))
    sums = (rows if systematic else 4 * rows ** 0.5) + 8
    exponent = 0.0 if g.dtype == torch.float32 else 2.0 ** -23 * f64(g.abs()).max((0, 1))
    tol = (2.0 ** -20 + exponent + sums * F) * (1 + U[dtype]) + U[dtype]
    floor = TINY[dtype] * np.prod(want.shape[:-1]) ** 0.5
    assert np.all(np.isfinite(got)), what
    excess = err - tol * size - floor
    worst = int(np.argmax(excess))
    assert excess[worst] <= 0, (f"{what}: gate {GATES[worst % len(GATES)]}: {err[worst] / size[worst]:.2e} of the channel, "
                                f"allowed {np.broadcast_to(tol, size.shape)[worst]:.2e}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("spread,constant", [(0.5, False), (0.0, False), (0.0, True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_gates_that_keep_a_state(shape, spread, constant, state, dtype):
    x, g, s = data(shape, dtype, spread, constant, state)
    reverse = shape[1] % 200 == 100
    ref = f64(x), f64(g), np.zeros((shape[0], shape[2])) if s is None else f64(s)
    h, before, last, parts = scan64(*ref, reverse)
    systematic = constant or state or shape[1] == 1
    for save in (False, True):
        got = sla.sla_gated_scan(x, g, s, reverse=reverse, save=save)
        check(got[0], h, g, shape[1], dtype, systematic, "h")
        check(got[1], last, g, shape[1], torch.float32, systematic, "final", parts)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    dh = torch.randn(*shape, generator=gen, device=DEV).to(dtype)
    dlast = torch.randn(shape[0], shape[2], generator=gen, device=DEV)
    want = back64(*ref[:2], before, f64(dh), f64(dlast), reverse)
    dx, dg, ds = sla.sla_gated_scan_backward(dh, x, g, got[2], dlast, s, reverse=reverse)
    check(dx, want[0], g, shape[1], dtype, True, "dx")
    check(ds, want[2], g, shape[1], torch.float32, True, "dstate", want[3])
    if not constant:  # (h - x of constant inputs is their difference's rounding where gates are closed)
        check(dg, want[1], g, shape[1], dtype, True, "dgate")
    if s is None and not constant:
        # without a state h is linear in x: sum dh h + sum dlast last = sum dx x, what the two calls say of one another
        left = (f64(dh) * f64(got[0])).sum((0, 1)) + (f64(dlast) * f64(got[1])).sum(0)
        terms = np.abs(f64(dh) * h).sum((0, 1)) + np.abs(f64(dlast) * last).sum(0) + np.abs(want[0] * ref[0]).sum((0, 1))
        right = (f64(dx) * ref[0]).sum((0, 1))
        tol = 2.0 ** -18 + 2 * shape[1] * F + 2 * U[dtype]
        floor = TINY[dtype] * (np.abs(f64(dh)) + np.abs(ref[0])).sum((0, 1))
        assert np.all(np.abs(left - right) <= tol * terms + floor)
    sla.sla_gated_ffn_check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_packed_sequences_that_keep_a_state(reverse, dtype):
    lengths = [300, 1, 0, 700, 255, 257, 2, 5000]
    marks = np.concatenate(([0], np.cumsum(lengths))).tolist()
    x, g, s = data((1, marks[-1], 51), dtype, 0.5, False, True)
    s = torch.randn(len(lengths), 51, device=DEV) * 1e-3
    offsets = torch.tensor(marks, device=DEV)
    h, last = sla.sla_gated_scan(x[0], g[0], s, offsets, reverse)
    for i, (p, q) in enumerate(zip(marks, marks[1:])):
        if p == q:
            assert torch.equal(last[i], s[i])
            continue
        want, _, end, parts = scan64(f64(x[:, p:q]), f64(g[:, p:q]), f64(s[i:i + 1]), reverse)
        check(h[None, p:q], want, g, q - p, dtype, True, "h")
        check(last[i:i + 1], end, g, q - p, torch.float32, True, "final", parts)


def test_one_path_of_a_million_rows():
    """A gate of 14 carries a state over a path of a million cells.  What a map takes from a state is right to the 2^-20 of 1 - a and
    a rounding a row, 128 F; the state itself goes through 16 spans, in each through 31 folds, 15 tiles, 8 warps and itself, and at the end
    through a warp's 16 rows, each a rounding: 16 * 55 F + 16 F."""
    allowed = (16 * 55 + 16 + 128) * F + 3 * 2.0 ** -20  # (over a factor of e^-3 at most)
    n, c = 1_000_000, 8
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    gates = torch.tensor([11.0, 12.0, 13.0, 14.0], device=DEV).repeat(2)
    g = gates.expand(n, c).contiguous()
    x = torch.zeros(n, c, device=DEV)
    x[:, :4] = torch.randn(n, 4, generator=gen, device=DEV)
    s = torch.zeros(1, c, device=DEV)
    s[:, 4:] = 1.0  # the last four channels: a state alone
    h, _ = sla.sla_gated_scan(x, g, s)
    at = torch.arange(1, n + 1, device=DEV, dtype=torch.float64)[:, None]
    want = torch.exp(at * torch.log1p(-1 / (1 + torch.exp(gates[4:].double()))))
    near = want > 0.05
    assert float(((h[:, 4:].double() - want).abs() / want)[near].max()) <= allowed
    a, b = torch.sigmoid(gates[:4].double()), torch.sigmoid(-gates[:4].double())
    # h of the inputs alone, blocks of 1000 rows side by side
    v = (b * x[:, :4].double()).view(1000, 1000, 4)
    rows = [v[:, 0]]
    for t in range(1, 1000):
        rows.append(a * rows[-1] + v[:, t])
    inside, carry, carries = torch.stack(rows, 1), torch.zeros(4, dtype=torch.float64, device=DEV), []
    for k in range(1000):
        carries.append(carry)
        carry = inside[k, -1] + a ** 1000 * carry
    power = a ** torch.arange(1, 1001, device=DEV, dtype=torch.float64)[:, None]
    want = (inside + power * torch.stack(carries)[:, None]).view(n, 4)
    err = ((h[:, :4].double() - want).norm(dim=0) / want.norm(dim=0)).max()
    assert float(err) <= allowed


def test_gradients_behind_an_input_that_stands_out():
    """The backward call forms the states again: one large input among small ones leaves its neighbours' gradients right."""
    for shape in ((1, 64, 64), (1, 700, 34), (760, 70, 2)):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(6)
        x, dh = (torch.randn(*shape, generator=gen, device=DEV) for _ in range(2))
        g = 12 + 0.5 * torch.randn(*shape, generator=gen, device=DEV)
        s = torch.randn(shape[0], shape[2], generator=gen, device=DEV)
        x[:, 3::24] = 1e4
        zero = torch.zeros_like(s)
        _, _, saved = sla.sla_gated_scan(x, g, s, save=True)
        _, dg, _ = sla.sla_gated_scan_backward(dh, x, g, saved, zero, s)
        x, g, dh = f64(x), f64(g), f64(dh)
        _, before, _, _ = scan64(x, g, f64(s))
        _, want, _, _ = back64(x, g, before, dh, f64(zero))
        # dgate = l (h - x) a (1 - a): errors of l and h are n F of the largest ones along the way, those of the rest 2^-20
        l = want / np.where(before == x, 1, before - x)  # with a (1 - a)
        ab = 1 / (1 + np.exp(g)) / (1 + np.exp(-g))
        parts = ab * np.abs(l / ab).max() * np.abs(before - x) + np.abs(l) * np.abs(before).max()
        assert np.all(np.abs(f64(dg) - want) <= (2.0 ** -19 + 4 * shape[1] * F) * parts)


def test_infinities_and_extremes():
    """Values next to the largest float32 of either sign, and gates at their ends."""
    big = 3e38
    x = torch.tensor([[big], [-big], [big], [-big]], device=DEV).repeat(1, 2)
    for gate in (-200.0, -3.0, 0.0, 3.0, 12.0, 200.0, float("inf"), -float("inf")):
        g = torch.full_like(x, gate)
        s = torch.full((1, 2), -big, device=DEV)
        h, _, saved = sla.sla_gated_scan(x, g, s, save=True)
        want = scan64(f64(x)[None], np.clip(f64(g), -700, 700)[None], f64(s))[0][0]
        assert np.all(np.abs(f64(h) - want) <= 2.0 ** -18 * big), gate
        dx, dg, ds = sla.sla_gated_scan_backward(torch.ones_like(x), x, g, saved, None, s)
        assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(ds).all()), gate
