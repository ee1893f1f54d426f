"""What becomes of a bounded wait that expires: the calls after it and the check report it, to every thread that was there."""
import threading

import pytest

from gpu_helpers import sla, torch
from test_gpu_dense import ffn_inputs

pytestmark = pytest.mark.gpu


def step():
    args = [t.requires_grad_() for t in ffn_inputs(40, 32, 48, 16, torch.bfloat16, True, seed=250)]
    return sla.gated_ffn(*args).sum()


def expire():
    sla.sla_test_expire_wait()
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def told():
    """Before and after each test this thread and autograd's know of everything."""
    def settle():
        for _ in range(2):
            try:
                sla.sla_gated_ffn_check()
                step().backward()
            except sla.SlaError:
                pass
        sla.sla_gated_ffn_check()
        step().backward()

    settle()
    yield
    torch.cuda.synchronize()
    settle()


def test_the_next_call_reports_it_once():
    args = ffn_inputs(40, 32, 48, 16, torch.bfloat16, True, seed=250)
    want = sla.sla_gated_ffn(*args)
    expire()
    with pytest.raises(sla.SlaError, match="TIMEOUT"):
        sla.sla_gated_ffn(*args)
    assert torch.equal(sla.sla_gated_ffn(*args), want)
    sla.sla_gated_ffn_check()


def test_the_check_waits_for_it_and_reports_it_once():
    sla.sla_test_expire_wait()
    sla.sla_test_expire_wait()
    with pytest.raises(sla.SlaError, match="TIMEOUT"):
        sla.sla_gated_ffn_check()
    sla.sla_gated_ffn_check()
    step()


def test_a_backward_call_reports_it():
    loss = step()
    expire()
    with pytest.raises(sla.SlaError, match="TIMEOUT"):
        loss.backward()


def test_every_thread_is_told_and_none_takes_anothers_report():
    met, expired, found = threading.Barrier(4), threading.Event(), []

    def work():
        sla.sla_gated_ffn_check()
        met.wait(60)
        assert expired.wait(60)
        for _ in range(2):
            try:
                sla.sla_gated_ffn_check()
                found.append("nothing")
            except sla.SlaError as e:
                found.append("timeout" if "TIMEOUT" in str(e) else str(e))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    met.wait(60)
    expire()
    expired.set()
    for t in threads:
        t.join()
    assert sorted(found) == ["nothing"] * 3 + ["timeout"] * 3
    with pytest.raises(sla.SlaError, match="TIMEOUT"):
        sla.sla_gated_ffn_check()
    # a thread that comes later has nothing to do with it
    late = []
    t = threading.Thread(target=lambda: late.append(sla.sla_gated_ffn_check()))
    t.start()
    t.join()
    assert late == [None]


def test_it_is_seen_from_a_graph():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        sla.sla_gated_ffn_check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sla.sla_test_expire_wait()
    sla.sla_gated_ffn_check()
    graph.replay()
    with pytest.raises(sla.SlaError, match="TIMEOUT"):
        sla.sla_gated_ffn_check()
