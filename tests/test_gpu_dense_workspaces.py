"""Workspaces that the caller brings: one that fits is used, one that is no dense memory of the device is refused."""
import pytest

from gpu_helpers import sla, torch, DEV
from test_gpu_dense import ffn_inputs, randn

from differentiable_sparse_iterative_gb300 import dense

pytestmark = pytest.mark.gpu


def test_workspaces_of_the_dense_operators():
    args = ffn_inputs(40, 100, 96, 50, torch.bfloat16, True, seed=240)
    dy = randn(40, 50, dtype=torch.bfloat16, seed=241)
    x = randn(30, 100, dtype=torch.float32, seed=242)
    _, mean, rstd = sla.sla_layernorm(x, stats=True)
    want, saved = sla.sla_gated_ffn(*args, save=True)
    calls = [lambda ws: sla.sla_gated_ffn(*args, workspace=ws),
             lambda ws: sla.sla_gated_ffn_backward(dy, *args[:3], saved, workspace=ws)[0],
             lambda ws: sla.sla_layernorm_backward(x, x, None, mean, rstd, workspace=ws)[0]]
    n = 1 << 24
    for call in calls:
        for bad, message in ((torch.empty(n, dtype=torch.uint8), "CUDA tensor"),
                             (torch.empty(n, dtype=torch.uint8).pin_memory(), "CUDA tensor"),
                             (torch.empty(1, dtype=torch.uint8, device=DEV).expand(n), "contiguous"),
                             (torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2], "contiguous")):
            with pytest.raises(ValueError, match=message):
                call(bad)
        own = torch.empty(n // 4, dtype=torch.float32, device=DEV)
        assert torch.equal(call(own), call(None))
        with pytest.raises(sla.SlaError):  # not on 256 bytes
            call(torch.empty(n, dtype=torch.uint8, device=DEV)[16:])
        assert torch.equal(call(torch.empty(256, dtype=torch.uint8, device=DEV)), call(None))  # too small: not used
    assert torch.equal(want, calls[0](None))
    assert dense._scratch(100, torch.device(DEV), None)[1] == 256


def test_saved_of_another_call_is_refused():
    args = ffn_inputs(40, 96, 64, 32, torch.bfloat16, False, seed=245)
    dy = randn(40, 32, dtype=torch.bfloat16, seed=246)
    _, saved = sla.sla_gated_ffn(*args, save=True)
    want = sla.sla_gated_ffn_backward(dy, *args[:3], saved)
    other = ffn_inputs(40, 64, 64, 32, torch.bfloat16, False, seed=247)
    _, theirs = sla.sla_gated_ffn(*other, save=True)
    assert theirs.numel() == saved.numel()  # nothing is kept of x and the weights: the width does not count
    half = ffn_inputs(40, 96, 64, 32, torch.float16, False, seed=248)
    for bad, what in ((theirs, {}), (saved, {"activation": "gelu"}),
                      (sla.sla_gated_ffn(*half, save=True)[1], {}), (torch.cat((saved, saved)), {})):
        with pytest.raises(ValueError, match="another activation"):
            sla.sla_gated_ffn_backward(dy, *args[:3], bad, **what)
    for kept in (saved, saved.clone()):
        got = sla.sla_gated_ffn_backward(dy, *args[:3], kept)
        assert all(p is None or torch.equal(p, q) for p, q in zip(got, want))
