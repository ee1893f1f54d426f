"""The device that a call runs with, without a GPU: tensors that say they are on another one, and a stand-in for the switch to it."""
import pytest

torch = pytest.importorskip("torch")

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402
from differentiable_sparse_iterative_gb300 import dense  # noqa: E402


class Elsewhere(torch.Tensor):
    """A tensor that says it is on cuda:1."""
    is_cuda = True

    def get_device(self):
        return 1


class Switched(Exception):
    pass


@pytest.fixture
def switch(monkeypatch):
    """cuda:0 is the current device, and a switch to another one raises."""
    def device(index):
        raise Switched(index)

    monkeypatch.setattr(dense, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)


def t(*shape):
    return torch.empty(*shape).as_subclass(Elsewhere)


CALLS = {
    "scan, no dh": lambda: sla.sla_gated_scan_backward(None, t(4, 8), t(4, 8), t(256), t(1, 8)),
    "scan, no dh, by keyword": lambda: sla.sla_gated_scan_backward(dh=None, x=t(4, 8), gate=t(4, 8), saved=t(256)),
    "scan, dh": lambda: sla.sla_gated_scan_backward(t(4, 8), t(4, 8), t(4, 8), t(256)),
    "scan forward": lambda: sla.sla_gated_scan(x=t(4, 8), gate=t(4, 8)),
    "norm, no dz": lambda: sla.sla_residual_norm_backward(None, t(4, 8), t(4, 8), t(4, 8), t(4, 4)),
    "norm, neither": lambda: sla.sla_residual_norm_backward(None, None, t(4, 8), t(4, 8), t(4, 4)),
    "norm, no dz, by keyword": lambda: sla.sla_residual_norm_backward(dy=t(4, 8), dz=None, block=t(4, 8), z=t(4, 8), stats=t(4, 4)),
    "norm, dz": lambda: sla.sla_residual_norm_backward(t(4, 8), None, t(4, 8), t(4, 8), t(4, 4)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_runs_on_its_tensors_device(name, switch):
    with pytest.raises(Switched) as e:
        CALLS[name]()
    assert e.value.args == (1,)


def test_a_call_on_the_current_device_switches_nothing(switch, monkeypatch):
    monkeypatch.setattr(dense, "_current_device", lambda: 1)
    seen = []
    call = dense._on_device_of_first(lambda first, second=None: seen.append((first, second)))
    call(None, t(2))
    call(t(2))
    call(None)
    call(None, torch.empty(2))  # a tensor on the CPU: refused inside of the call
    assert len(seen) == 4
