"""Training steps of the gated feed-forward block on inputs laid out in every way that a call may read or copy them.

A forward call leaves copies of some operands to its backward call.  Whatever the layout, the backward call must find
them written: every buffer that the binding allocates starts out as NaN here.  Tolerances: those of test_gpu_dense.py.
"""
import pytest

from gpu_helpers import sla, torch
from test_gpu_dense import FFN_TOL, TYPES, ffn64, ffn_inputs, randn, rel

from differentiable_sparse_iterative_gb300 import dense

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def nan_memory(monkeypatch):
    def empty(*args, **kw):
        t = torch.empty(*args, **kw)
        return t.fill_(255 if t.dtype == torch.uint8 else float("nan"))  # bytes of 255 are NaN in all three types

    monkeypatch.setattr(dense, "_empty", empty)


def sliced(t, ld, offset):
    """t's values in columns [offset, offset + width) of an array with rows ld apart."""
    big = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=t.device)
    big[:, offset:offset + t.shape[1]] = t
    return big[:, offset:offset + t.shape[1]]


# tokens, width, hidden, out; distance between the rows of x and of dy (0: dense), first column
LAYOUTS = [((300, 250, 96, 64), 256, 0, 0), ((40, 250, 683, 131), 256, 136, 0), ((17, 100, 104, 20), 104, 24, 0),
           ((300, 250, 96, 64), 264, 72, 8), ((129, 250, 96, 64), 251, 65, 1), ((64, 65, 100, 50), 80, 56, 3),
           ((300, 64, 100, 1), 0, 0, 0), ((300, 65, 683, 1), 0, 0, 0), ((130, 250, 100, 1), 256, 8, 0),
           ((40, 64, 1, 8), 0, 0, 0), ((40, 1, 1, 1), 8, 8, 0), ((33, 1, 64, 64), 0, 0, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,ldx,lddy,offset", LAYOUTS)
def test_ffn_training_step_of_any_layout(shape, ldx, lddy, offset, dtype):
    args = ffn_inputs(*shape, dtype, True, seed=200)
    dy = randn(shape[0], shape[3], dtype=dtype, seed=206)
    leaves = [t.double().requires_grad_() for t in args]
    ref = ffn64(*leaves, "silu")
    grads = torch.autograd.grad(ref, leaves, dy.double())
    x = sliced(args[0], ldx, offset) if ldx else args[0]
    dy = sliced(dy, lddy, offset) if lddy else dy
    y, saved = sla.sla_gated_ffn(x, *args[1:], save=True)
    got = sla.sla_gated_ffn_backward(dy, x, *args[1:3], saved, want_grad_bias=True)
    assert rel(y, ref.detach()) <= FFN_TOL[dtype]
    for name, g, r in zip(("dx", "dw_in", "dw_out", "db_in", "db_out"), got, grads):
        assert rel(g, r) <= FFN_TOL[dtype], (name, rel(g, r))
    # the differentiable entry, with x as a view of the wider array
    leaves = [x.detach(), *(t.clone() for t in args[1:])]
    for t in leaves:
        t.requires_grad_()
    got = torch.autograd.grad(sla.gated_ffn(*leaves), leaves, dy)
    for name, g, r in zip(("x", "w_in", "w_out", "b_in", "b_out"), got, grads):
        assert rel(g, r) <= FFN_TOL[dtype], (name, rel(g, r))
