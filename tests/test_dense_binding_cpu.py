"""The dense operators' Python entries, with the calls behind them replaced (no GPU needed)."""
import inspect

import pytest

torch = pytest.importorskip("torch")

import torch.autograd.forward_ad as fwad  # noqa: E402

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402
from differentiable_sparse_iterative_gb300 import dense  # noqa: E402


@pytest.fixture
def plain(monkeypatch):
    """The two forward calls as a few torch operations on CPU tensors."""
    def layernorm(x, weight=None, bias=None, eps=1e-5, y=None, stats=False):
        y = torch.nn.functional.layer_norm(x, x.shape[-1:], weight, bias, eps)
        return (y, x[..., 0].clone(), x[..., 0].clone()) if stats else y

    def gated_ffn(x, w_in, w_out, b_in=None, b_out=None, activation="silu", y=None, save=False, workspace=None):
        g, u = torch.nn.functional.linear(x, w_in, b_in).chunk(2, -1)
        y = torch.nn.functional.linear(torch.nn.functional.silu(g) * u, w_out, b_out)
        return (y, torch.zeros(1, dtype=torch.uint8)) if save else y

    monkeypatch.setattr(dense, "sla_layernorm", layernorm)
    monkeypatch.setattr(dense, "sla_gated_ffn", gated_ffn)


def _calls():
    """(call, its arguments)"""
    gen = torch.Generator().manual_seed(1)
    x, w, b = torch.randn(3, 8, generator=gen), torch.randn(8, generator=gen), torch.randn(8, generator=gen)
    w_in, w_out = torch.randn(12, 8, generator=gen), torch.randn(5, 6, generator=gen)
    b_in, b_out = torch.randn(12, generator=gen), torch.randn(5, generator=gen)
    return [(sla.layer_norm, [x, w, b]), (sla.gated_ffn, [x, w_in, w_out, b_in, b_out])]


@pytest.mark.parametrize("grad", [True, False])
def test_a_forward_mode_tangent_is_refused_not_dropped(plain, grad):
    for call, args in _calls():
        call(*args)
        for i, t in enumerate(args):
            with fwad.dual_level(), torch.set_grad_enabled(grad):
                moved = list(args)
                moved[i] = fwad.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError):
                    call(*moved)
            with pytest.raises(RuntimeError):  # as any node without a rule for torch.func
                torch.func.jvp(lambda v: call(*args[:i], v, *args[i + 1:]), (t,), (torch.ones_like(t),))


def test_the_node_is_taken_for_gradients_alone(plain):
    for call, args in _calls():
        assert call(*args).grad_fn is None
        for i, t in enumerate(args):
            moved = list(args)
            moved[i] = t.clone().requires_grad_()
            assert call(*moved).grad_fn is not None
            with torch.no_grad():
                assert call(*moved).grad_fn is None
            with fwad.dual_level():
                assert call(*args).grad_fn is None


class _Cuda:
    """What the check of a workspace looks at, of a CUDA tensor."""
    is_cuda = True

    def __init__(self, index, numel, contiguous=True):
        self.index, self.size, self.contiguous, self.device = index, numel, contiguous, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def numel(self):
        return self.size

    def element_size(self):
        return 4

    def is_contiguous(self):
        return self.contiguous


def test_a_workspace_that_is_not_dense_memory_of_the_device_is_refused():
    dev = torch.device("cuda", 0)
    for ws, message in ((torch.empty(1 << 12, dtype=torch.uint8), "CUDA tensor"), (torch.empty(8), "CUDA tensor"),
                        (_Cuda(1, 1 << 12), "on cuda:0"), (_Cuda(0, 1 << 12, contiguous=False), "contiguous")):
        with pytest.raises(ValueError, match=message):
            dense._scratch(1024, dev, ws)
    good = _Cuda(0, 256)
    assert dense._scratch(1024, dev, good) == (good, 1024)


def test_a_solver_workspace_that_is_not_dense_memory_of_the_device_is_refused():
    dev = torch.device("cuda", 0)
    for ws, message in ((torch.empty(1 << 12, dtype=torch.uint8), "CUDA tensor"), (_Cuda(1, 1 << 12), "on cuda:0"),
                        (_Cuda(0, 1 << 12, contiguous=False), "contiguous")):
        with pytest.raises(ValueError, match=message):
            sla._scratch(1024, dev, ws)
    good = _Cuda(0, 256)
    assert sla._scratch(1024, dev, good) is good
    assert sla._scratch(100, torch.device("cpu"), None).numel() == 256


@pytest.fixture
def two_devices(monkeypatch):
    """Two devices of which 0 is current; the list gets what is done under which."""
    state = {"current": 0, "seen": []}

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *_):
            state["current"] = self.before

    monkeypatch.setattr(dense, "_current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(dense, "_stream", lambda index: 1000 + index)
    return state


def test_a_call_runs_on_its_tensors_device(two_devices):
    # each entry's first look at its tensors is recorded in place of the call
    for call, name in ((sla.sla_layernorm, "x"), (sla.sla_layernorm_backward, "dy"), (sla.sla_gated_ffn, "x"),
                       (sla.sla_gated_ffn_backward, "dy")):
        body = call.__wrapped__

        def record(*args, **kw):
            two_devices["seen"].append(two_devices["current"])

        record.__signature__ = inspect.signature(body)
        wrapped = dense._on_device_of_first(record)
        two_devices["seen"].clear()
        wrapped(_Cuda(0, 1))
        wrapped(_Cuda(1, 1))
        wrapped(**{name: _Cuda(1, 1)})
        wrapped(torch.ones(2))  # refused by the call itself
        assert two_devices["seen"] == [0, 1, 1, 0] and two_devices["current"] == 0


def test_the_check_reads_the_device_that_it_is_asked_about(two_devices, monkeypatch):
    class Lib:
        def sla_gated_ffn_check(self, stream):
            two_devices["seen"].append((two_devices["current"], stream))
            return 0

    monkeypatch.setattr(dense, "_library", Lib())
    sla.sla_gated_ffn_check()
    sla.sla_gated_ffn_check(1)
    assert two_devices["seen"] == [(0, 1000), (1, 1001)] and two_devices["current"] == 0
