"""Forward-mode derivatives are refused by the dense operators as solve() refuses them, on the GPU's own path."""
import pytest

import torch.autograd.forward_ad as fwad

from gpu_helpers import sla, torch
from test_gpu_dense import ffn_inputs, randn

pytestmark = pytest.mark.gpu


def test_tangents_are_refused():
    x, w_in, w_out, _, _ = ffn_inputs(20, 32, 16, 8, torch.float32, False, seed=230)
    w = randn(32, dtype=torch.float32, seed=231)
    with fwad.dual_level():
        for i in range(3):
            args = [x, w_in, w_out]
            args[i] = fwad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(NotImplementedError):
                sla.gated_ffn(*args)
        for args in ((fwad.make_dual(x, torch.ones_like(x)), w), (x, fwad.make_dual(w, torch.ones_like(w)))):
            with pytest.raises(NotImplementedError):
                sla.layer_norm(*args)
        assert sla.layer_norm(x, w).grad_fn is None
