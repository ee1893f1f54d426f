"""Argument checks of the dense operators' C entry points and binding (no GPU needed)."""
import ctypes

import pytest

from differentiable_sparse_iterative_gb300 import _abi, build as sla_build

torch = pytest.importorskip("torch")

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402

P = 0x10000  # never dereferenced: every case is rejected before any CUDA call
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    sla_build.build()
    if torch.cuda.is_available():
        pytest.skip("fake-pointer ABI checks run only on machines without a GPU")
    return _abi.load()


def _ffn(tokens=8, width=16, hidden=32, out=16, dtype=3, activation=0):
    f = _abi.sla_ffn()
    f.tokens, f.width, f.hidden, f.out, f.dtype, f.activation = tokens, width, hidden, out, dtype, activation
    return ctypes.byref(f)


def test_layernorm_arguments(lib):
    def fwd(rows=4, width=16, dtype=3, pt=3, x=P, ldx=16, w=P, b=P, eps=1e-5, y=P, mean=P, rstd=P):
        return lib.sla_layernorm(rows, width, dtype, pt, x, ldx, w, b, eps, y, mean, rstd, None)

    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=(1 << 24) + 1), dict(dtype=1),
                dict(dtype=4), dict(pt=2), dict(pt=1), dict(x=None), dict(y=None), dict(ldx=15), dict(x=P + 1),
                dict(w=P + 1), dict(b=P + 1), dict(mean=P + 2), dict(rstd=P + 2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert fwd(**bad) == _abi.SLA_INVALID_ARG, bad
    assert fwd(rows=0, x=None, y=None) == _abi.SLA_OK

    def bwd(rows=4, width=16, dtype=3, pt=0, dy=P, lddy=16, x=P, ldx=16, w=P, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P,
            n=BIG):
        return lib.sla_layernorm_backward(rows, width, dtype, pt, dy, lddy, x, ldx, w, mean, rstd, dx, dw, db, ws, n,
                                          None)

    for bad in (dict(rows=-1), dict(width=0), dict(dtype=1), dict(pt=2), dict(dy=None), dict(x=None), dict(lddy=3),
                dict(ldx=3), dict(mean=None), dict(rstd=None), dict(dx=P + 1), dict(dw=P + 2), dict(db=P + 2),
                dict(ws=None), dict(ws=P + 8)):
        assert bwd(**bad) == _abi.SLA_INVALID_ARG, bad
    assert bwd(n=8) == _abi.SLA_WORKSPACE_TOO_SMALL
    assert bwd(dx=None, dw=None, db=None, ws=None, n=0) == _abi.SLA_OK  # nothing wanted
    need = lib.sla_layernorm_backward_workspace_bytes
    assert need(-1, 8, 3) == need(8, 0, 3) == need(8, 8, 1) == 0
    assert need(1000, 64, 3) >= 2 * 64 * 4 and need(1000, 64, 0) % 256 == 0


def test_ffn_arguments(lib):
    def fwd(f=None, x=P, ldx=16, w_in=P, b_in=None, w_out=P, b_out=None, y=P, saved=P, sn=BIG, ws=P, wn=BIG):
        return lib.sla_gated_ffn(f or _ffn(), x, ldx, w_in, b_in, w_out, b_out, y, saved, sn, ws, wn, None)

    shapes = (dict(tokens=-1), dict(tokens=1 << 31), dict(width=0), dict(hidden=0), dict(out=0),
              dict(hidden=(1 << 24) + 1), dict(dtype=1), dict(dtype=7), dict(activation=-1), dict(activation=4))
    for bad in shapes:
        f = _ffn(**bad)
        assert fwd(f) == _abi.SLA_INVALID_ARG, bad
        assert lib.sla_gated_ffn_saved_bytes(f) == lib.sla_gated_ffn_workspace_bytes(f) == 0
        assert lib.sla_gated_ffn_backward_workspace_bytes(f) == 0
    for bad in (dict(x=None), dict(x=P + 1), dict(ldx=15), dict(w_in=None), dict(w_out=None), dict(w_in=P + 1),
                dict(b_in=P + 1), dict(b_out=P + 1), dict(y=None), dict(saved=P + 16), dict(ws=None), dict(ws=P + 16)):
        assert fwd(**bad) == _abi.SLA_INVALID_ARG, bad
    assert fwd(sn=16) == _abi.SLA_WORKSPACE_TOO_SMALL and fwd(wn=16) == _abi.SLA_WORKSPACE_TOO_SMALL
    assert fwd(_ffn(tokens=0), x=None, y=None) == _abi.SLA_OK

    def bwd(f=None, dy=P, lddy=16, x=P, ldx=16, w_in=P, w_out=P, saved=P, sn=BIG, grads=(P,) * 5, ws=P, wn=BIG):
        return lib.sla_gated_ffn_backward(f or _ffn(), dy, lddy, x, ldx, w_in, w_out, saved, sn, *grads, ws, wn, None)

    for bad in (dict(dy=None), dict(lddy=1), dict(x=None), dict(ldx=1), dict(w_in=None), dict(w_out=None),
                dict(saved=None), dict(saved=P + 8), dict(ws=None), dict(grads=(P + 1, P, P, P, P)),
                dict(grads=(P, P, P, P, P + 1))):
        assert bwd(**bad) == _abi.SLA_INVALID_ARG, bad
    assert bwd(sn=16) == _abi.SLA_WORKSPACE_TOO_SMALL and bwd(wn=16) == _abi.SLA_WORKSPACE_TOO_SMALL


def test_cpu_tensors_are_refused():
    sla_build.build()
    x, w_in, w_out = torch.ones(2, 8), torch.ones(8, 8), torch.ones(3, 4)
    for call in (lambda: sla.layer_norm(x), lambda: sla.sla_layernorm(x), lambda: sla.gated_ffn(x, w_in, w_out),
                 lambda: sla.sla_gated_ffn(x, w_in, w_out),
                 lambda: sla.sla_layernorm_backward(x, x, None, x[:, 0], x[:, 0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_layernorm_workspace_covers_every_class_of_rows(lib):
    # rows of odd widths are dealt to blocks in whole sets of up to 8 classes, so that a few rows can have more
    # blocks than there are rows: the partial sums of all of them have to fit
    for rows in (1, 9, 17, 20, 100, 1209, 1215, 5000):
        for width, dtype, classes in ((8191, 3, 8), (8193, 2, 8), (4095, 0, 4), (4100, 3, 2)):
            blocks = min(1216 // classes * classes, -(-rows // classes) * classes)
            assert lib.sla_layernorm_backward_workspace_bytes(rows, width, dtype) >= blocks * 2 * width * 4
