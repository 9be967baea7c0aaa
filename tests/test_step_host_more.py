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
        monkeypatch.setattr(P, "_done", self.done)
        monkeypatch.setattr(P._Prepared, "_launch", lambda call: self.log.append(("launch", self.stream)))

    def wait_event(self, event):
        self.log.append(("wait", self.stream))

    def done(self, event, wait):
        if wait:
            self.log.append(("finish", self.stream))
        return wait or self.ready

    def call(self, capture=0):
        c = P._Counted.__new__(P._Counted)
        c._name, c._index, c._made_on = "call", 0, self.stream
        c._capture, c._zeroed, c._first = capture, None if capture else self, True
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
    m.ready = False                      # is not asked again
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
        assert m.log == [("finish", 2), ("launch", 2), ("launch", 2)]


def test_the_two_helpers_refuse_null():
    assert P._capture_id(None, None) == 1 and P._event_done(None, 0, None) == 1 and P._event_done(1, 1, None) == 1
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


def test_what_a_call_writes_is_marked_as_changed(monkeypatch):
    """An operator that has saved a tensor for its backward pass is told that a call wrote over it, as torch's own writes tell it."""
    from sparse_attention_csa2_gb300 import paged
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 1)
    status = [0]
    call = paged._Prepared()
    mine, theirs, kept = torch.ones(4), torch.ones(4), torch.ones(4)
    call._bind(lambda ref, stream: status[0], C.c_int(), torch.device("cuda", 0), (mine,), (kept,), (theirs, None))
    w = torch.ones(4, requires_grad=True)
    products = [(t * w).sum() for t in (mine, theirs, kept)]
    call._launch()
    for p in products[:2]:
        with pytest.raises(RuntimeError, match="inplace"):
            p.backward()
    products[2].backward()
    with torch.inference_mode():
        call._written = (torch.ones(4),)   # has no version
        call._launch()
    status[0] = 1
    before = theirs._version
    call._written = (theirs,)
    with pytest.raises(S.CSA2Error):
        call._launch()
    assert theirs._version == before


def test_every_call_that_writes_what_it_is_given_says_so(monkeypatch):
    from sparse_attention_csa2_gb300 import paged
    seen = {}

    class Stop(Exception):
        pass

    def bind(self, call, args, device, mine, keep, written=()):
        seen[type(self).__name__] = (*mine, *written)
        raise Stop

    monkeypatch.setattr(paged._Prepared, "_bind", bind)
    for module in (paged, P):
        monkeypatch.setattr(module, "_on", lambda t, name, device=None: 0)
        monkeypatch.setattr(module, "_dense", lambda t, name, dtype, shape, device=None: 0)
    monkeypatch.setattr(P._Counted, "_workspace", lambda self, n, device: setattr(self, "_wsp", None) or (0, 0))
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    x, r, to, out = (torch.zeros(4, 64) for _ in range(4))
    table, q = i32(2, 3), torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache = paged.PageCache.empty(3, 2, 16, 64, device="cpu")
    o16, q_out = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros_like(q)
    experts = S.ExpertWeights(torch.zeros(3, 32, 64, dtype=torch.bfloat16), torch.zeros(3, 64, 16, dtype=torch.bfloat16))
    status = i32(1)
    for name, make, written in (
            ("AddNorm", lambda: S.AddNorm(x, residual=r), (r,)),
            ("AddNorm", lambda: S.AddNorm(x, residual=r, residual_out=to, out=out), (to, out)),
            ("MoEExperts", lambda: S.MoEExperts(o16, i32(4, 2), torch.zeros(4, 2), experts, out=out, dev_status=status), (out, status)),
            ("PagePlan", lambda: S.PagePlan(i32(2), i32(2), table, i32(5), 16, 8), (table,)),
            ("PageWriter", lambda: S.PageWriter(cache, q, q, i32(3), i32(2), i32(4), table), tuple(cache)),
            ("RopeAxes", lambda: S.RopeAxes(q, torch.zeros(4, dtype=torch.int64), out=q_out), (q_out,)),
            ("PagedAttn", lambda: S.PagedAttn(q, cache, i32(3), i32(2), table, 1.0, out=q_out), (q_out,))):
        with pytest.raises(Stop):
            make()
        assert all(any(t is s for s in seen[name]) for t in written), name
