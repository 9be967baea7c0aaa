"""Prepared calls that follow attention, on a machine without a GPU: where their counters are zero."""
import ctypes as C

import pytest
import torch

S = pytest.importorskip("sparse_attention_csa2_gb300")
from sparse_attention_csa2_gb300 import step as P  # noqa: E402


class Machine:
    """A device whose current stream, captures and events are numbers."""

    def __init__(self, monkeypatch):
        self.stream, self.captures, self.log, self.ready = 1, {}, [], False
        monkeypatch.setattr(P, "_raw_stream", lambda index: self.stream)
        monkeypatch.setattr(P, "_capture_of", lambda stream: self.captures.get(stream, 0))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(self.captures.get(self.stream)))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda: self)
        monkeypatch.setattr(P, "_finish_event", lambda e: self.log.append(("finish", e)) or 0)
        monkeypatch.setattr(P._Prepared, "_launch", lambda call: self.log.append(("launch", self.stream)))
        self.cuda_event = 7

    def wait_event(self, event):
        self.log.append(("wait", self.stream))

    def query(self):
        assert not self.captures.get(self.stream), "an event is not asked during a capture"
        return self.ready

    def call(self, capture=0):
        c = P._Counted.__new__(P._Counted)
        c._name, c._index, c._made_on = "call", 0, self.stream
        c._capture, c._zeroed = capture, None if capture else self
        return c


def test_a_call_made_within_a_capture_runs_in_that_alone(monkeypatch):
    m = Machine(monkeypatch)
    m.captures[1] = 5
    call = m.call(capture=5)
    call._launch()
    m.stream, m.captures[2] = 2, 5       # a stream that joined the capture
    call._launch()
    for other in (6, 0):                 # another capture; none
        m.captures = {1: other}
        for m.stream in (1, 2):
            with pytest.raises(RuntimeError, match="capture"):
                call._launch()
    assert m.log == [("launch", 1), ("launch", 2)]


def test_a_call_comes_behind_its_zeros(monkeypatch):
    m = Machine(monkeypatch)
    call = m.call()
    call._launch()                       # behind them anyway
    m.stream = 2
    call._launch()
    m.ready = True
    call._launch()
    m.ready = None                       # is not asked again
    call._launch()
    assert m.log == [("launch", 1), ("wait", 2), ("launch", 2), ("launch", 2), ("launch", 2)]


def test_a_captured_call_has_its_zeros(monkeypatch):
    for made_on in (1, 2):               # a graph runs behind nothing, also one that was captured on the stream of the zeros
        m = Machine(monkeypatch)
        m.stream = made_on
        call = m.call()
        m.stream, m.captures = 2, {2: 9}
        call._launch()
        call._launch()
        assert m.log == [("finish", 7), ("launch", 2), ("launch", 2)]


def test_the_two_helpers_refuse_null():
    assert P._capture_id(None, None) == 1 and P._finish_event(None) == 1
    assert P._capture_id.argtypes[1] is C.POINTER(C.c_uint64)


def test_dual_tensors_are_refused():
    """Forward mode sets no requires_grad, and is on under torch.no_grad()."""
    fwd = torch.autograd.forward_ad
    x, i32, f32 = torch.zeros(4, 64), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2)
    up, down = torch.zeros(3, 32, 64, dtype=torch.bfloat16), torch.zeros(3, 64, 16, dtype=torch.bfloat16)
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        calls = [lambda: S.add_norm(dual(x)), lambda: S.add_norm(x, dual(x[0])), lambda: S.add_norm(x, residual=dual(x)),
                 lambda: S.route_experts(x, dual(x), 2), lambda: S.route_experts(x, x, 2, bias=dual(torch.zeros(4))),
                 lambda: S.moe_experts(dual(x.bfloat16()), i32, f32, S.ExpertWeights(up, down)),
                 lambda: S.moe_experts(x.bfloat16(), i32, dual(f32), S.ExpertWeights(up, down)),
                 lambda: S.moe_experts(x.bfloat16(), i32, f32, S.ExpertWeights(up, dual(down))),
                 lambda: S.sample_tokens(dual(x), torch.zeros(4)), lambda: S.sample_tokens(x, torch.zeros(4), temperature=dual(torch.ones(4))),
                 lambda: S.rope_axes(dual(x[:, None]), torch.zeros(4, dtype=torch.int64))]
        for call in calls:
            with pytest.raises(ValueError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
                call()
        for call in (lambda: S.add_norm(fwd.unpack_dual(dual(x)).primal), lambda: S.add_norm(x)):
            with pytest.raises(ValueError, match="CUDA"):   # on to the next check
                call()
