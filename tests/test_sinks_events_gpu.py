"""The timing events of a backward pass with sinks: all of dK and dV lies between theirs."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import Geometry, draw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_dk_and_dv_are_complete_at_their_stop_event():
    """Copies on another stream that wait for that event alone, beside a query-major pass of hundreds of microseconds."""
    g = Geometry("BNSD", 1, 8, 128, S_q=8192, S_kv=8192, N_kv=1, scale=128 ** -0.5, sparse_mode=4, pre_tokens=2000,
                 next_tokens=0, sink_tokens=140)
    inp = draw(g, 3)
    q, k, v, dy = (t.to(DEV) for t in (inp.q, inp.k, inp.v, inp.dy))
    out, smax, ssum = swa.forward(g, q, k, v)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    ws = torch.empty(swa.swa_backward_workspace_size(swa.Params(g)), dtype=torch.uint8, device=DEV)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
    for e in events:  # their handles exist from here on
        e.record()
    early = [torch.empty_like(t) for t in (dk, dv)]
    side = torch.cuda.Stream()
    for again in range(4):
        for t in (dk, dv):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        swa.swa_set_timing_events([e.cuda_event for e in events])
        try:
            swa.backward(g, q, k, v, dy, out, smax, ssum, dq=dq, dk=dk, dv=dv, workspace=ws)
        finally:
            swa.swa_set_timing_events()
        side.wait_event(events[3])
        with torch.cuda.stream(side):
            for t, x in zip(early, (dk, dv)):
                t.copy_(x)
        torch.cuda.synchronize()
        for t, x in zip(early, (dk, dv)):
            assert not torch.isnan(x).any() and torch.equal(t, x), again
