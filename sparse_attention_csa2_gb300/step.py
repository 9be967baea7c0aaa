"""What follows attention in a decode step: the norm with the residual's addition (and an 8-bit output), the
router and its experts, and the choice of a token from the logits.

    norm = add_norm(attn_out, gain, residual=stream)                       # stream += attn_out, norm.out
    route = route_experts(norm.out, w_router, k=6, bias=bias, score="sigmoid")
    y = moe_experts(norm.out, route.ids, route.weights, experts, n_shared=1)
    token, logprob = sample_tokens(logits, u, temperature=t, top_k=k, top_p=p, min_p=m)

Each call exists as a class that binds its tensors once (as the paged cache's calls do) and is then run by
calling the object, for decode loops and for capture into a CUDA graph.  Running one object on two streams at
once races on its outputs and workspace.  A router or experts object made within a capture belongs to that graph:
calls outside it, or in another capture, are refused.  These calls record no autograd graph: tensors whose gradient torch
would track are refused outside torch.no_grad(), and forward mode's dual tensors everywhere.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional

import torch

from . import _check, _f32, _i32, _i64, _sig, _sz, _vp
from .paged import _TYPES, _Prepared, _dense, _int, _no_tangent, _on, _raw_stream


class AddNormArgs(C.Structure):
    _fields_ = [("n_rows", _i32), ("dim", _i32), ("x_dtype", _i32), ("sum_dtype", _i32), ("out_dtype", _i32),
                ("gain_dtype", _i32), ("group", _i32), ("x", _vp), ("x_row", _i64), ("residual", _vp),
                ("residual_row", _i64), ("sum", _vp), ("sum_row", _i64), ("gain", _vp), ("gain_offset", _f32),
                ("eps", _f32), ("out", _vp), ("out_row", _i64), ("codes", _vp), ("scales", _vp)]


class RouteArgs(C.Structure):
    _fields_ = [("tokens", _i32), ("dim", _i32), ("experts", _i32), ("k", _i32), ("x_dtype", _i32), ("w_dtype", _i32),
                ("score", _i32), ("normalize", _i32), ("scale", _f32), ("x", _vp), ("x_row", _i64), ("w", _vp),
                ("bias", _vp), ("ids", _vp), ("weights", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class MoEArgs(C.Structure):
    _fields_ = [("tokens", _i32), ("k", _i32), ("experts", _i32), ("n_shared", _i32), ("dim", _i32), ("inner", _i32),
                ("x_codes", _i32), ("w_codes", _i32), ("out_dtype", _i32), ("limit", _f32), ("x", _vp), ("x_row", _i64),
                ("x_scale", _vp), ("ids", _vp), ("weights", _vp), ("up", _vp), ("down", _vp), ("up_scale", _vp),
                ("down_scale", _vp), ("out", _vp), ("out_row", _i64), ("workspace", _vp), ("workspace_bytes", _sz),
                ("dev_status", _vp), ("form", _i32)]


class SampleArgs(C.Structure):
    _fields_ = [("n_rows", _i32), ("vocab", _i32), ("dtype", _i32), ("logits", _vp), ("row", _i64), ("u", _vp),
                ("temperature", _vp), ("top_k", _vp), ("top_p", _vp), ("min_p", _vp), ("token", _vp), ("logprob", _vp)]


COUNTER_BYTES = 65536
FORMS = {None: 0, "few": 1, "many": 2}
SCORES = {"softmax": 0, "sigmoid": 1, "sqrtsoftplus": 2}
_add_norm = _sig("csa2_add_norm", [C.POINTER(AddNormArgs), _vp], C.c_int)
_route_ws = _sig("csa2_route_workspace_size", [C.POINTER(RouteArgs)], _sz)
_route = _sig("csa2_route", [C.POINTER(RouteArgs), _vp], C.c_int)
_moe_ws = _sig("csa2_moe_workspace_size", [C.POINTER(MoEArgs)], _sz)
_moe = _sig("csa2_moe", [C.POINTER(MoEArgs), _vp], C.c_int)
_moe_waits = _sig("csa2_selftest_moe_waits", [C.POINTER(MoEArgs), _i32, _vp], C.c_int)
_sample = _sig("csa2_sample", [C.POINTER(SampleArgs), _vp], C.c_int)
_capture_id = _sig("csa2_capture_id", [_vp, C.POINTER(C.c_uint64)], C.c_int)
_event_done = _sig("csa2_event_done", [_vp, _i32, C.POINTER(_i32)], C.c_int)


# ------------------------------------------------------------------ checks
def _forward_only(name, *tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{name} records no gradient: call it under torch.no_grad() or with detached tensors")
    _no_tangent(name, *tensors)


def _rows(t, name, device=None, shape=None):
    """Address and row stride of a [rows, dim] tensor whose last dimension is dense."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be [rows, dim]" + (f" of {tuple(shape)}" if shape is not None else "") + f", got {tuple(t.shape)}")
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32")
    if t.shape[1] > 1 and t.stride(1) != 1 and t.numel():
        raise ValueError(f"{name} must be dense in its last dimension")
    return _on(t, name, device), t.stride(0) if t.shape[0] > 1 else 0


def _capture_of(stream) -> int:
    """A number of the graph capture that a stream is in, 0 outside."""
    of = C.c_uint64()
    _check(_capture_id(stream, C.byref(of)), "csa2_capture_id")
    return of.value


def _done(event, wait: bool) -> bool:
    """Whether an event's work has ended, on wish after a wait; unlike event.query() also while any thread captures a graph."""
    done = _i32()
    _check(_event_done(event.cuda_event, wait, C.byref(done)), "csa2_event_done")
    return bool(done.value)


class _Counted(_Prepared):
    """A prepared call whose workspace begins with counters that are zero between calls."""

    def _workspace(self, nbytes, device):
        self._wsp = torch.empty(max(int(nbytes), COUNTER_BYTES), dtype=torch.uint8, device=device)
        with torch.cuda.device(device):
            self._wsp[:COUNTER_BYTES].zero_()
            # in a capture the zeros are the graph's; otherwise until they are known to be there, calls come behind them
            self._capture = _capture_of(_raw_stream(device.index)) if torch.cuda.is_current_stream_capturing() else 0
            self._zeroed = None if self._capture else torch.cuda.current_stream().record_event()
            self._first = True
        return self._wsp.data_ptr(), self._wsp.numel()

    def _launch(self):
        if self._capture or self._zeroed is not None:
            self._behind_zeros()
        super()._launch()

    def _behind_zeros(self):
        if self._capture:
            if _capture_of(_raw_stream(self._index)) != self._capture:
                raise RuntimeError(f"{self._name}: made within a graph capture, whose runs alone have its counters at zero")
            return
        first, self._first = self._first, False
        capturing, elsewhere = torch.cuda.is_current_stream_capturing(), _raw_stream(self._index) != self._made_on
        if first and not capturing and not elsewhere:
            return  # the usual way of an object that is run once
        if _done(self._zeroed, capturing):  # a graph may run on any stream, behind nothing
            self._zeroed = None
        elif elsewhere:
            torch.cuda.current_stream().wait_event(self._zeroed)


# ------------------------------------------------------------------ norm
class AddNorm(_Prepared):
    """A prepared csa2_add_norm call: rows x [T, dim] (bf16, fp16 or fp32; rows may be strided), added to
    `residual` where there is one (x's type or fp32; the sum goes to `residual_out`, by default back into
    residual), divided by their root mean square and multiplied by weight [dim] + gain_offset.

    .out: the rows in `out_dtype` (x's type by default; with quant_group only on request, by out_dtype or out);
    .codes, .scales: with quant_group, E4M3 codes [T, dim] uint8 and their fp32 scales, [T] for quant_group 0
    or [T, dim / quant_group] (16, 32, 64, 128, 256): value = code * scale; .residual_out: the sum."""
    _name = "csa2_add_norm"

    def __init__(self, x, weight=None, residual=None, eps: float = 1e-6, gain_offset: float = 0.0, residual_out=None,
                 out_dtype=None, quant_group=None, out=None):
        _forward_only("add_norm", x, weight, residual, residual_out, out)
        dev = x.device
        a = AddNormArgs()
        a.x, a.x_row = _rows(x, "x")
        T, D = x.shape
        a.n_rows, a.dim, a.x_dtype = T, D, _TYPES[x.dtype]
        mine = []
        if residual is None:
            if residual_out is not None:
                raise ValueError("residual_out without a residual")
        else:
            if residual_out is None:
                residual_out = residual
            a.residual, a.residual_row = _rows(residual, "residual", dev, x.shape)
            a.sum, a.sum_row = _rows(residual_out, "residual_out", dev, x.shape)
            if residual.dtype not in (x.dtype, torch.float32) or residual_out.dtype != residual.dtype:
                raise ValueError("residual must be of x's type or float32, and residual_out of residual's")
            a.sum_dtype = _TYPES[residual.dtype]
        if weight is not None:
            if weight.dtype not in _TYPES:
                raise ValueError("weight must be bfloat16, float16 or float32")
            a.gain, a.gain_dtype = _dense(weight, "weight", weight.dtype, (D,), dev), _TYPES[weight.dtype]
        a.gain_offset, a.eps = float(gain_offset), float(eps)
        if out is None and (quant_group is None or out_dtype is not None):
            out = torch.empty((T, D), dtype=out_dtype or x.dtype, device=dev)
            mine.append(out)
        if out is not None:
            if out_dtype is not None and out.dtype != out_dtype:
                raise ValueError("out has another type than out_dtype")
            a.out, a.out_row = _rows(out, "out", dev, x.shape)
            a.out_dtype = _TYPES[out.dtype]
        self.codes = self.scales = None
        if quant_group is not None:
            a.group = g = _int(quant_group, "quant_group")
            if g not in (0, 16, 32, 64, 128, 256) or (g and D % g):
                raise ValueError("quant_group must be 0, 16, 32, 64, 128 or 256 and divide the rows")
            self.codes = torch.empty((T, D), dtype=torch.uint8, device=dev)
            self.scales = torch.empty((T, D // g) if g else (T,), dtype=torch.float32, device=dev)
            a.codes, a.scales = self.codes.data_ptr(), self.scales.data_ptr()
            mine += [self.codes, self.scales]
        self.out, self.residual_out = out, residual_out
        self._bind(_add_norm, a, dev, tuple(mine), (x, weight, residual, residual_out, out), (residual_out, out))

    def __call__(self):
        self._run()
        return self


def add_norm(x, weight=None, residual=None, eps: float = 1e-6, gain_offset: float = 0.0, residual_out=None, out_dtype=None,
             quant_group=None, out=None):
    """Root-mean-square norm of x (+ residual) (see AddNorm); returns the AddNorm after running it."""
    return AddNorm(x, weight, residual, eps, gain_offset, residual_out, out_dtype, quant_group, out)()


# ------------------------------------------------------------------ experts
class ExpertRouter(_Counted):
    """A prepared csa2_route call: the k experts of each row of x [T, dim] (bf16, fp16 or fp32; rows may be strided)
    by the products with w [experts, dim] (x's type or fp32) and `score` ("softmax", "sigmoid", "sqrtsoftplus"):
    those with the largest score + bias [experts] fp32.

    .ids [T, k] int32, in falling order; .weights [T, k] fp32: their scores, over their sum if `normalize`, times
    `scale`."""
    _name = "csa2_route"

    def __init__(self, x, w, k: int, bias=None, score: str = "softmax", normalize: bool = True, scale: float = 1.0):
        _forward_only("route_experts", x, w, bias)
        if score not in SCORES:
            raise ValueError(f"score is one of {', '.join(SCORES)}")
        dev = x.device
        a = RouteArgs()
        a.x, a.x_row = _rows(x, "x")
        T, D = x.shape
        if w.dim() != 2 or w.dtype not in (x.dtype, torch.float32):
            raise ValueError("w must be [experts, dim] of x's type or float32")
        E = w.shape[0]
        a.w = _dense(w, "w", w.dtype, (E, D), dev)
        a.bias = None if bias is None else _dense(bias, "bias", torch.float32, (E,), dev)
        a.tokens, a.dim, a.experts, a.k = T, D, E, _int(k, "k")
        a.x_dtype, a.w_dtype, a.score = _TYPES[x.dtype], _TYPES[w.dtype], SCORES[score]
        a.normalize, a.scale = bool(normalize), float(scale)
        self.ids = torch.empty((T, a.k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, a.k), dtype=torch.float32, device=dev)
        a.ids, a.weights = self.ids.data_ptr(), self.weights.data_ptr()
        a.workspace, a.workspace_bytes = self._workspace(_route_ws(C.byref(a)), dev)
        self._bind(_route, a, dev, (self.ids, self.weights, self._wsp), (x, w, bias))

    def __call__(self):
        self._run()
        return self


def route_experts(x, w, k: int, bias=None, score: str = "softmax", normalize: bool = True, scale: float = 1.0):
    """The experts of each token and their weights (see ExpertRouter); returns the ExpertRouter after running it."""
    return ExpertRouter(x, w, k, bias, score, normalize, scale)()


class ExpertWeights(NamedTuple):
    """Weights of a layer's experts, the shared ones behind the routed ones: up [experts, 2 inner, dim] with the gate's
    rows before the up projection's, down [experts, dim, inner]; bf16, or uint8 E4M3 codes with up_scale
    [experts, 2 inner] and down_scale [experts, dim] fp32: value = code * scale."""
    up: torch.Tensor
    down: torch.Tensor
    up_scale: Optional[torch.Tensor] = None
    down_scale: Optional[torch.Tensor] = None


class MoEExperts(_Counted):
    """A prepared csa2_moe call: out [T, dim] (bf16, or out_dtype float32) of x [T, dim] (bf16, or uint8 E4M3 codes with
    x_scale [T] fp32, as add_norm gives them; rows may be strided) through the experts ids [T, k] int32 (-1: none) with
    weights [T, k] fp32, and through the last `n_shared` of `experts` with weight 1.  `limit` clamps the gate from above
    and the up projection on both sides.  For up to 512 tokens (a decode step, drafts): the weights of the experts that
    are met are what it reads.  `form` ("few", "many") overrides the choice by the tokens per expert, for tests and tuning.
    dev_status [1] int32 tells of ids out of range, which are left out, and of waits that ran out, with which out is NaN."""
    _name = "csa2_moe"

    def __init__(self, x, ids, weights, experts: ExpertWeights, n_shared: int = 0, limit=None, x_scale=None, out_dtype=None,
                 out=None, dev_status=None, form=None):
        _forward_only("moe_experts", x, weights, x_scale, out, *experts)
        dev = x.device
        a = MoEArgs()
        if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.uint8) or (x.shape[1] > 1 and x.stride(1) != 1 and x.numel()):
            raise ValueError("x must be [tokens, dim], bfloat16 or uint8 codes, dense in its last dimension")
        T, D = x.shape
        a.x, a.x_row = _on(x, "x"), x.stride(0) if T > 1 else 0
        a.x_codes = x.dtype == torch.uint8
        if (x_scale is not None) != bool(a.x_codes):
            raise ValueError("x_scale goes with uint8 codes")
        a.x_scale = None if x_scale is None else _dense(x_scale, "x_scale", torch.float32, (T,), dev)
        if ids.dim() != 2:
            raise ValueError("ids must be [tokens, k]")
        k = ids.shape[1]
        a.ids = _dense(ids, "ids", torch.int32, (T, k), dev)
        a.weights = _dense(weights, "weights", torch.float32, (T, k), dev)
        up, down, up_scale, down_scale = experts
        if up.dim() != 3 or up.shape[1] % 2 or up.dtype not in (torch.bfloat16, torch.uint8):
            raise ValueError("experts.up must be [experts, 2 inner, dim], bfloat16 or uint8 codes")
        n, F = up.shape[0], up.shape[1] // 2
        a.up = _dense(up, "experts.up", up.dtype, (n, 2 * F, D), dev)
        a.down = _dense(down, "experts.down", up.dtype, (n, D, F), dev)
        a.w_codes = up.dtype == torch.uint8
        if any((s is not None) != bool(a.w_codes) for s in (up_scale, down_scale)):
            raise ValueError("up_scale and down_scale go with uint8 codes")
        if a.w_codes:
            a.up_scale = _dense(up_scale, "experts.up_scale", torch.float32, (n, 2 * F), dev)
            a.down_scale = _dense(down_scale, "experts.down_scale", torch.float32, (n, D), dev)
        a.tokens, a.k, a.dim, a.inner, a.n_shared = T, k, D, F, _int(n_shared, "n_shared")
        if n <= a.n_shared:
            raise ValueError("experts must hold routed experts before the shared ones")
        a.experts = n - a.n_shared
        a.limit = float("inf") if limit is None else float(limit)
        if out is None:
            out = torch.empty((T, D), dtype=out_dtype or torch.bfloat16, device=dev)
        if out.dtype not in (torch.bfloat16, torch.float32) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must be bfloat16 or float32")
        a.out, a.out_row = _rows(out, "out", dev, (T, D))
        a.out_dtype = _TYPES[out.dtype]
        self.out = out
        a.dev_status = None if dev_status is None else _dense(dev_status, "dev_status", torch.int32, (1,), dev)
        if form not in FORMS:
            raise ValueError('form is "few", "many" or None')
        a.form = FORMS[form]
        a.workspace, a.workspace_bytes = self._workspace(_moe_ws(C.byref(a)), dev)
        self._bind(_moe, a, dev, (out, self._wsp), (x, ids, weights, experts, x_scale, dev_status), (dev_status,))

    def __call__(self):
        self._run()
        return self.out


def moe_experts(x, ids, weights, experts: ExpertWeights, n_shared: int = 0, limit=None, x_scale=None, out_dtype=None, out=None,
                dev_status=None, form=None):
    """The sum of each token's experts (see MoEExperts)."""
    return MoEExperts(x, ids, weights, experts, n_shared, limit, x_scale, out_dtype, out, dev_status, form)()


def selftest_moe_waits(call: MoEExperts, tries: int) -> None:
    """Runs a prepared call (with a dev_status) whose waits give up after `tries` tries (csa2_selftest_moe_waits): its
    status then reads ETIMEOUT and its output is NaN."""
    with torch.cuda.device(call._device):
        _check(_moe_waits(call._ref, int(tries), _raw_stream(call._index)), "csa2_selftest_moe_waits")


# ------------------------------------------------------------------ sampling
class TokenSampler(_Prepared):
    """A prepared csa2_sample call: a token of each row of logits [rows, vocab] (bf16, fp16 or fp32; rows may be strided)
    by the random number u [rows] fp32 in [0, 1).  temperature, top_p, min_p [rows] fp32 and top_k [rows] int32 are each
    row's own, None: 1 and no cut; a temperature of 0 is greedy, top_k 0, top_p 1 and min_p 0 cut nothing.

    .token [rows] int64 (-1 where no logit is above -infinity); .logprob [rows] fp32, of the token among the kept."""
    _name = "csa2_sample"

    def __init__(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
        _forward_only("sample_tokens", logits, u, temperature, top_p, min_p)
        dev = logits.device
        a = SampleArgs()
        a.logits, a.row = _rows(logits, "logits")
        n, a.vocab = logits.shape
        a.n_rows, a.dtype = n, _TYPES[logits.dtype]
        a.u = _dense(u, "u", torch.float32, (n,), dev)
        for name, t, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                               ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
            setattr(a, name, None if t is None else _dense(t, name, dtype, (n,), dev))
        self.token = torch.empty(n, dtype=torch.int64, device=dev)
        self.logprob = torch.empty(n, dtype=torch.float32, device=dev)
        a.token, a.logprob = self.token.data_ptr(), self.logprob.data_ptr()
        self._bind(_sample, a, dev, (self.token, self.logprob), (logits, u, temperature, top_k, top_p, min_p))

    def __call__(self):
        self._run()
        return self.token, self.logprob


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """A token of each row of logits and its log-probability among the kept ones (see TokenSampler)."""
    return TokenSampler(logits, u, temperature, top_k, top_p, min_p)()
