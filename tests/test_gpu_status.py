"""The status call of a chain, after work on a stream that does not wait for the
null stream."""
import pytest

from gpu_util import make_matrix, qg, to_dev, torch
from skinny_gemm_q4_gb300 import synth

pytestmark = pytest.mark.gpu


def test_chain_status_waits_for_every_stream(monkeypatch):
    """A wait that the host made run out (half a second, in a launch on a side
    stream) is in the error word when the status call, made at once, returns."""
    t = torch()
    M = K = 2560
    h = [make_matrix(qg.Q4_K, M, K, seed=i)[0] for i in range(2)]
    x = to_dev(synth.activations(1, K, seed=1, stream=1))
    y = [t.empty((1, M), dtype=t.float16, device="cuda") for _ in range(2)]
    calls = qg.make_calls([
        (qg.CALL_RUN, [h[0].h], x.data_ptr(), 1, [y[0].data_ptr()], qg.OUT_F16, None),
        (qg.CALL_RUN, [h[1].h], y[0].data_ptr(), 1, [y[1].data_ptr()], qg.OUT_F16, None)])
    ch = qg.Chain(qg.CHAIN_PERSISTENT)
    ch.run(calls)
    assert ch.status() == 0
    side = t.cuda.Stream()
    monkeypatch.setenv("QGEMV_FAULT_INJECT", "chain_publish")
    ch.run(calls, stream=side)
    monkeypatch.delenv("QGEMV_FAULT_INJECT")
    assert ch.status(clear=True) & 4
    assert ch.status() == 0
