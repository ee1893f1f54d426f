"""The linear layer, the residual norm and the gated scan without a GPU: C argument checks, sizes, and the Python entries."""
import ctypes

import pytest

from differentiable_sparse_iterative_gb300 import _abi, build as sla_build

torch = pytest.importorskip("torch")

import torch.autograd.forward_ad as fwad  # noqa: E402

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402
from differentiable_sparse_iterative_gb300 import dense, scan  # noqa: E402

P = 0x10000  # never dereferenced: every case is rejected before any CUDA call
BIG = 1 << 40
BAD, SMALL, OK = _abi.SLA_INVALID_ARG, _abi.SLA_WORKSPACE_TOO_SMALL, _abi.SLA_OK


@pytest.fixture(scope="module")
def lib():
    sla_build.build()
    if torch.cuda.is_available():
        pytest.skip("fake-pointer ABI checks run only on machines without a GPU")
    return _abi.load()


def layer(tokens=20, width=16, out=24, dtype=3, act=0):
    return ctypes.byref(_abi.sla_layer(tokens, width, out, dtype, act))


def test_linear_arguments(lib):
    def fwd(f=None, x=P, ldx=16, w=P, b=None, r=None, ldr=24, y=P, saved=P, sn=BIG, ws=P, wn=BIG):
        return lib.sla_linear(f or layer(), x, ldx, w, b, r, ldr, y, saved, sn, ws, wn, None)

    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(width=0), dict(out=0), dict(out=(1 << 24) + 1), dict(dtype=1),
                dict(dtype=7), dict(act=-1), dict(act=5)):
        f = layer(**bad)
        assert fwd(f) == BAD, bad
        assert lib.sla_linear_saved_bytes(f) == lib.sla_linear_workspace_bytes(f) == 0
        assert lib.sla_linear_backward_workspace_bytes(f) == 0
    for bad in (dict(x=None), dict(x=P + 1), dict(ldx=15), dict(w=None), dict(w=P + 1), dict(b=P + 1), dict(r=P + 1),
                dict(r=P, ldr=23), dict(y=None), dict(y=P + 1), dict(saved=P + 16), dict(ws=None), dict(ws=P + 16)):
        assert fwd(**bad) == BAD, bad
    assert fwd(sn=16) == SMALL and fwd(wn=16) == SMALL
    assert fwd(layer(tokens=0), x=None, y=None, ws=P) == OK

    def bwd(f=None, dy=P, lddy=24, x=P, ldx=16, w=P, saved=P, sn=BIG, grads=(P,) * 3, ws=P, wn=BIG):
        return lib.sla_linear_backward(f or layer(), dy, lddy, x, ldx, w, saved, sn, *grads, ws, wn, None)

    for bad in (dict(dy=None), dict(lddy=1), dict(x=None), dict(ldx=1), dict(w=None), dict(saved=None), dict(saved=P + 8),
                dict(ws=None), dict(grads=(P + 1, P, P)), dict(grads=(P, P + 1, P)), dict(grads=(P, P, P + 1))):
        assert bwd(**bad) == BAD, bad
    assert bwd(sn=16) == SMALL and bwd(wn=16) == SMALL
    assert bwd(grads=(None,) * 3) == OK  # nothing wanted
    assert lib.sla_linear_saved_bytes(layer(act=_abi.SLA_ACT_NONE)) == 0  # nothing to keep
    assert lib.sla_linear_saved_bytes(layer(act=_abi.SLA_ACT_NONE, dtype=0)) > 0
    assert lib.sla_linear_workspace_bytes(layer(tokens=3)) == 0


def resnorm(rows=4, width=16, dtype=3, pt=3, norm=0, post=1, act=0, reserved=0, eps=1e-5):
    return ctypes.byref(_abi.sla_resnorm(rows, width, dtype, pt, norm, post, act, reserved, eps))


def test_residual_norm_arguments(lib):
    def fwd(n=None, f=P, ldf=16, z=P, ldz=16, g=None, ldg=16, params=(P,) * 5, zo=P, y=P, stats=P):
        return lib.sla_residual_norm(n or resnorm(), f, ldf, z, ldz, g, ldg, *params, zo, y, stats, None)

    shapes = (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=(1 << 24) + 1), dict(dtype=1), dict(pt=2),
              dict(norm=2), dict(post=2), dict(act=3), dict(act=-1), dict(reserved=1), dict(eps=-1.0), dict(eps=float("nan")))
    for bad in shapes:
        assert fwd(resnorm(**bad)) == BAD, bad
        assert lib.sla_residual_norm_backward_workspace_bytes(resnorm(**bad)) == 0
    for bad in (dict(f=None), dict(f=P + 1), dict(ldf=15), dict(ldf=1 << 29), dict(z=None), dict(ldz=3), dict(g=P + 1),
                dict(g=P, ldg=2), dict(zo=None), dict(y=P + 1), dict(stats=P + 4),
                *[dict(params=tuple(P + 1 if i == k else P for i in range(5))) for k in range(5)]):
        assert fwd(**bad) == BAD, bad
    assert fwd(resnorm(rows=0), f=None, z=None, zo=None, y=None) == OK

    def bwd(n=None, dz=P, lddz=16, dy=P, lddy=16, f=P, ldf=16, z=P, ldz=16, g=P, ldg=16, params=(P,) * 4, stats=P,
            grads=(P,) * 8, ws=P, wn=BIG):
        return lib.sla_residual_norm_backward(n or resnorm(), dz, lddz, dy, lddy, f, ldf, z, ldz, g, ldg, *params, stats,
                                              *grads, ws, wn, None)

    for bad in (dict(dz=P + 1), dict(lddz=3), dict(dy=P + 1), dict(lddy=3), dict(f=None), dict(z=None), dict(g=None),
                dict(stats=None), dict(stats=P + 8), dict(ws=None), dict(ws=P + 8),
                *[dict(grads=tuple(P + 1 if i == k else P for i in range(8))) for k in range(8)]):
        assert bwd(**bad) == BAD, bad
    assert bwd(wn=16) == SMALL
    assert bwd(grads=(None,) * 8, ws=None, wn=0) == OK
    # rows of odd widths are dealt to blocks in whole sets of up to 8 classes: the partial sums of all of them have to fit
    for rows in (1, 9, 100, 5000):
        for width, groups, blocks in ((33, 32, 304), (1001, 2, 304), (8183, 1, 152)):  # rows a block takes at a time, blocks at most
            need = lib.sla_residual_norm_backward_workspace_bytes(resnorm(rows=rows, width=width))
            for classes in (1, 2, 4, 8):
                sets = min(blocks // classes, -(-(-(-rows // classes)) // groups))
                assert need >= 5 * 4 * width * max(1, sets) * classes


def a_scan(rows=600, channels=64, sequences=2, offsets=None, ot=0, dtype=3, reverse=0, outside=0):
    return ctypes.byref(_abi.sla_scan(rows, channels, sequences, offsets, ot, dtype, reverse, outside))


def test_scan_arguments(lib):
    def fwd(s=None, x=P, ldx=64, g=P, ldg=64, state=P, h=P, final=P, saved=P, sn=BIG, ws=P, wn=BIG):
        return lib.sla_gated_scan(s or a_scan(), x, ldx, g, ldg, state, h, final, saved, sn, ws, wn, None)

    def bwd(s=None, dh=P, lddh=64, dfinal=P, x=P, ldx=64, g=P, ldg=64, state=P, saved=P, sn=BIG, grads=(P,) * 3, ws=P, wn=BIG):
        return lib.sla_gated_scan_backward(s or a_scan(), dh, lddh, dfinal, x, ldx, g, ldg, state, saved, sn, *grads, ws, wn,
                                           None)

    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(channels=0), dict(channels=(1 << 24) + 1), dict(sequences=-1),
                dict(sequences=7), dict(sequences=0), dict(dtype=1), dict(reverse=2), dict(outside=2),
                dict(offsets=P, ot=2), dict(offsets=P + 2), dict(offsets=P + 4, ot=1),
                dict(rows=(1 << 31) - 2, channels=1 << 20)):
        s = a_scan(**bad)
        assert fwd(s) == BAD and bwd(s) == BAD, bad
        assert lib.sla_gated_scan_saved_bytes(s) == lib.sla_gated_scan_workspace_bytes(s) == 0
    common = (dict(x=None), dict(x=P + 1), dict(ldx=63), dict(ldx=1 << 28), dict(g=None), dict(ldg=1), dict(state=P + 2),
              dict(saved=P + 8), dict(ws=None), dict(ws=P + 8))
    for bad in (*common, dict(h=None), dict(final=P + 1)):
        assert fwd(**bad) == BAD, bad
    for bad in (*common, dict(dh=P + 1), dict(lddh=3), dict(dfinal=P + 1), dict(saved=None), dict(grads=(P + 1, P, P)),
                dict(grads=(P, P + 1, P)), dict(grads=(P, P, P + 2))):
        assert bwd(**bad) == BAD, bad
    assert fwd(sn=16) == fwd(wn=16) == bwd(sn=16) == bwd(wn=16) == SMALL
    assert bwd(grads=(None,) * 3) == OK
    assert lib.sla_gated_scan_workspace_bytes(a_scan(rows=64, sequences=64)) == 0  # single steps need none
    assert lib.sla_gated_scan_workspace_bytes(a_scan(rows=64, sequences=64, offsets=P)) == 0  # nor what one block holds
    assert lib.sla_gated_scan_workspace_bytes(a_scan()) > 0
    assert lib.sla_gated_scan_saved_bytes(a_scan()) >= 600 // 16 * 64 * 4


def test_cpu_tensors_are_refused():
    sla_build.build()
    x, w = torch.ones(4, 8), torch.ones(3, 8)
    for call in (lambda: sla.linear(x, w), lambda: sla.sla_linear(x, w), lambda: sla.residual_norm(x, x),
                 lambda: sla.sla_residual_norm(x, x), lambda: sla.gated_scan(x, x), lambda: sla.sla_gated_scan(x, x),
                 lambda: sla.sla_gated_scan_backward(x, x, x, x), lambda: sla.sla_linear_backward(x, x, w, x),
                 lambda: sla.sla_residual_norm_backward(x, x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.fixture
def plain(monkeypatch):
    """The forward calls as a few torch operations on CPU tensors."""
    def linear(x, weight, bias=None, residual=None, activation="none", y=None, save=False, workspace=None):
        y = torch.nn.functional.linear(x, weight, bias) + (0 if residual is None else residual)
        return (y, torch.zeros(1, dtype=torch.uint8)) if save else y

    def residual_norm(block, z, gate=None, scale=None, post_weight=None, post_bias=None, weight=None, bias=None, norm="layer",
                      post_norm=True, next_norm=True, gate_activation="none", eps=1e-5, stats=False):
        z = z + block.sum() * sum(p.sum() for p in (gate, scale, post_weight, post_bias, weight, bias) if p is not None)
        return (z, z.clone(), z[:, :1]) if stats else (z, z.clone())

    def gated_scan(x, gate, state=None, offsets=None, reverse=False, h=None, final=None, save=False, workspace=None):
        h, final = x * gate, (torch.zeros(1, x.shape[-1]) if state is None else state.clone())
        return (h, final, torch.zeros(1, dtype=torch.uint8)) if save else (h, final)

    monkeypatch.setattr(dense, "sla_linear", linear)
    monkeypatch.setattr(dense, "sla_residual_norm", residual_norm)
    monkeypatch.setattr(scan, "sla_gated_scan", gated_scan)


def calls():
    """(call, its arguments, whether several results come back)"""
    gen = torch.Generator().manual_seed(1)

    def r(*shape):
        return torch.randn(*shape, generator=gen)

    return [(sla.linear, [r(3, 8), r(5, 8), r(5), r(3, 5)]),
            (sla.residual_norm, [r(3, 8), r(3, 8), r(3, 8), r(8), r(8), r(8), r(8), r(8)]),
            (sla.gated_scan, [r(3, 8), r(3, 8), r(1, 8)])]


@pytest.mark.parametrize("grad", [True, False])
def test_a_forward_mode_tangent_is_refused_not_dropped(plain, grad):
    for call, args in calls():
        call(*args)
        for i, t in enumerate(args):
            with fwad.dual_level(), torch.set_grad_enabled(grad):
                moved = list(args)
                moved[i] = fwad.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError):
                    call(*moved)


def test_the_node_is_taken_for_gradients_alone(plain):
    def first(out):
        return out if isinstance(out, torch.Tensor) else out[0]

    for call, args in calls():
        assert first(call(*args)).grad_fn is None
        for i, t in enumerate(args):
            moved = list(args)
            moved[i] = t.clone().requires_grad_()
            assert first(call(*moved)).grad_fn is not None
            with torch.no_grad():
                assert first(call(*moved)).grad_fn is None
