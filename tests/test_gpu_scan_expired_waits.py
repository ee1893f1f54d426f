"""The gated scan's bounded waits: what a block waits for is withheld, and the wait runs out after a tenth of a millisecond.

Nothing faults: every block that waits gives up once, the launch ends, and the next call reports it.
"""
import time

import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

CLOCKS = 200_000


def data(sequences, rows, channels, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    x, g, dh = (torch.randn(sequences, rows, channels, generator=gen, device=DEV).to(dtype) for _ in range(3))
    return x, g, dh, torch.randn(sequences, channels, generator=gen, device=DEV)


def ends_soon(call):
    torch.cuda.synchronize()
    start = time.monotonic()
    call()
    torch.cuda.synchronize()
    return time.monotonic() - start < 1.0  # one wait of every block in turn, not one for every tile


@pytest.fixture(autouse=True)
def normal_waits_afterwards():
    yield
    sla.sla_test_set_scan_wait(0, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("sequences,rows,channels", [(1, 60_000, 64), (1, 20_001, 130), (3, 700, 33)])
def test_a_wait_that_runs_out_is_reported(sequences, rows, channels, reverse, dtype):
    x, g, dh, s = data(sequences, rows, channels, dtype)
    h, final, saved = sla.sla_gated_scan(x, g, s, reverse=reverse, save=True)
    grads = sla.sla_gated_scan_backward(dh, x, g, saved, s, s, reverse=reverse)
    sla.sla_gated_ffn_check()

    def forward():
        return sla.sla_gated_scan(x, g, s, reverse=reverse)

    def backward():
        return sla.sla_gated_scan_backward(dh, x, g, saved, s, s, reverse=reverse)

    for call in (forward, backward):
        sla.sla_test_set_scan_wait(1, CLOCKS)
        assert ends_soon(call)
        sla.sla_test_set_scan_wait(0, 0)
        with pytest.raises(sla.SlaError) as e:
            call()
        assert e.value.status == sla._abi.SLA_TIMEOUT
        again = call()  # told once; and right again
        want = (h, final) if call is forward else grads
        assert all(torch.equal(p, q) for p, q in zip(again, want))
    sla.sla_gated_ffn_check()


def test_what_waits_for_nothing_is_not_held_up():
    """One tile, and a warp's walks: no waits."""
    for shape in ((1, 100, 64), (800, 300, 64)):
        x, g, dh, s = data(*shape, torch.float16)
        want = sla.sla_gated_scan(x, g, s)
        sla.sla_test_set_scan_wait(1, CLOCKS)
        got = sla.sla_gated_scan(x, g, s)
        sla.sla_test_set_scan_wait(0, 0)
        sla.sla_gated_ffn_check()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_replayed_call_that_runs_out_is_reported():
    x, g, dh, s = data(1, 30_000, 64, torch.bfloat16)
    want = sla.sla_gated_scan(x, g, s)
    torch.cuda.synchronize()
    sla.sla_test_set_scan_wait(1, CLOCKS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sla.sla_gated_scan(x, g, s)
    sla.sla_test_set_scan_wait(0, 0)
    sla.sla_gated_ffn_check()  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    with pytest.raises(sla.SlaError):
        sla.sla_gated_ffn_check()
    assert all(torch.equal(p, q) for p, q in zip(sla.sla_gated_scan(x, g, s), want))
