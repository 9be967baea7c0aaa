"""Paged 8-bit cache of a grouped-query attention layer: page tables and slot maps from request
lengths, rotary positions with several axes, the cache writer and attention over the cache.

One serving step is four calls on torch's current stream, none of which reads a length back:

    plan = page_plan(ctx_len, new_len, table, free_pages, page_size, max_rows)
    rope_axes(q, pos, sections=(16, 24, 24), out=q); rope_axes(k, pos, sections=(16, 24, 24), out=k)
    write_pages(cache, k, v, plan.row_start, plan.kv_len, plan.seq_of_row, table)
    out = paged_attn(q, cache, plan.row_start, plan.kv_len, table, softmax_scale=128 ** -0.5)

``plan.slot`` is also what ``write_records`` takes as destination rows.  Each call exists as a class
that binds its tensors once (as ``DecodeLayer`` does) and is then run by calling the object: for
decode loops and for capture into a CUDA graph.  Running one object on two streams at once races on
its outputs and workspace.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

from . import (_check, _f32, _i32, _i64, _lib, _sig, _sz, _vp, _ws)

T_BF16, T_F16, T_F32 = range(3)
ROPE_AXES_MAX_PAIRS = 128
_TYPES = {torch.bfloat16: T_BF16, torch.float16: T_F16, torch.float32: T_F32}


class PagePlanArgs(C.Structure):
    _fields_ = [("ctx_len", _vp), ("new_len", _vp), ("n_seq", _i32), ("page_size", _i32), ("table", _vp),
                ("table_cols", _i32), ("free_pages", _vp), ("n_free", _i32), ("max_rows", _i32), ("row_start", _vp),
                ("kv_len", _vp), ("seq_of_row", _vp), ("pos", _vp), ("slot", _vp), ("n_taken", _vp),
                ("dev_status", _vp)]


class RopeAxesArgs(C.Structure):
    _fields_ = [("n_tokens", _i32), ("n_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("x", _vp),
                ("x_row", _i64), ("x_head", _i64), ("out", _vp), ("out_row", _i64), ("out_head", _i64), ("pos", _vp),
                ("n_axes", _i32), ("rot_first", _i32), ("rot_dim", _i32), ("half_pairs", _i32), ("inverse", _i32),
                ("theta", _f32), ("axis_of_pair", C.c_uint8 * ROPE_AXES_MAX_PAIRS)]


class WritePagesArgs(C.Structure):
    _fields_ = [("n_rows", _i32), ("n_seq", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("n_pages", _i32), ("table_cols", _i32), ("dtype", _i32), ("k", _vp), ("k_row", _i64),
                ("k_head", _i64), ("v", _vp), ("v_row", _i64), ("v_head", _i64), ("row_start", _vp), ("kv_len", _vp),
                ("seq_of_row", _vp), ("table", _vp), ("k_codes", _vp), ("v_codes", _vp), ("k_scale", _vp),
                ("v_scale", _vp), ("dev_status", _vp)]


class PagedAttnArgs(C.Structure):
    _fields_ = [("n_rows", _i32), ("n_seq", _i32), ("heads", _i32), ("kv_heads", _i32), ("head_dim", _i32),
                ("page_size", _i32), ("n_pages", _i32), ("table_cols", _i32), ("q_dtype", _i32), ("out_dtype", _i32),
                ("q", _vp), ("q_row", _i64), ("q_head", _i64), ("row_start", _vp), ("kv_len", _vp), ("table", _vp),
                ("k_codes", _vp), ("v_codes", _vp), ("k_scale", _vp), ("v_scale", _vp), ("softmax_scale", _f32),
                ("window", _i32), ("sink", _vp), ("out", _vp), ("workspace", _vp), ("workspace_bytes", _sz),
                ("dev_status", _vp)]


_page_plan = _sig("csa2_page_plan", [C.POINTER(PagePlanArgs), _vp], C.c_int)
_rope_axes = _sig("csa2_rope_axes", [C.POINTER(RopeAxesArgs), _vp], C.c_int)
_write_pages = _sig("csa2_write_pages", [C.POINTER(WritePagesArgs), _vp], C.c_int)
_paged_attn_ws = _sig("csa2_paged_attn_workspace_size", [C.POINTER(PagedAttnArgs)], _sz)
_paged_attn = _sig("csa2_paged_attn", [C.POINTER(PagedAttnArgs), _vp], C.c_int)
_paged_waits = _sig("csa2_selftest_paged_waits", [C.POINTER(PagedAttnArgs), _i32, _vp], C.c_int)


_raw_stream = torch._C._cuda_getCurrentRawStream  # a device's current stream as a number


# ------------------------------------------------------------------ checks
def _dense(t, name, dtype, shape, device=None):
    """The address of a dense tensor of the given type and shape on the call's device."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return _on(t, name, device)


def _on(t, name, device=None):
    if any(n >= 2 ** 31 for n in t.shape):  # the C struct would cut it
        raise ValueError(f"{name} must be below 2^31 in every dimension, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _int(v, name):
    """A number that the C struct holds whole."""
    v = int(v)
    if not 0 <= v < 2 ** 31:
        raise ValueError(f"{name} must be at least 0 and below 2^31, got {v}")
    return v


def _heads(t, name, device=None):
    """Address and strides of a [rows, heads, dim] tensor whose last dimension is dense."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, dim]")
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32")
    if t.shape[2] > 1 and t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name} must be dense in its last dimension")
    row = t.stride(0) if t.shape[0] > 1 else 0  # the stride of an axis of one is never taken
    head = t.stride(1) if t.shape[1] > 1 else 0
    return _on(t, name, device), row, head


class _Prepared:
    """A call with its tensors bound: runs on the current stream of its tensors' device."""
    _name = ""

    def _bind(self, call, args, device, mine, keep):
        self._call, self._args, self._device = call, args, device
        self._ref = C.byref(args)
        self._mine, self._keep = mine, keep
        self._index = device.index
        self._made_on = _raw_stream(self._index)
        self._alone = torch.cuda.device_count() == 1

    def _run(self):
        # a decode step is made of such calls of a few microseconds each: no stream objects, no context
        # managers on the usual way
        if not self._alone and torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._device):
                return self._launch()
        return self._launch()

    def _launch(self):
        raw = _raw_stream(self._index)
        if raw != self._made_on:  # outputs and workspace outlive this stream's work when they are freed
            stream = torch.cuda.current_stream()
            for t in self._mine:
                t.record_stream(stream)
        status = self._call(self._ref, raw)
        if status:
            _check(status, self._name)


# ------------------------------------------------------------------ page plan
class PagePlan(_Prepared):
    """A prepared csa2_page_plan call.  ctx_len and new_len [n] int32 (tokens in the cache, tokens to
    come), table [n, columns] int32 with the cached tokens' pages, free_pages [F] int32.  Running it
    fills in the new tokens' pages in `table` and writes

    row_start [n + 1], kv_len [n], n_taken [1] int32, and for each of max_rows rows seq_of_row int32,
    pos and slot int64 (-1 behind the last sequence)."""
    _name = "csa2_page_plan"

    def __init__(self, ctx_len, new_len, table, free_pages, page_size: int, max_rows: int, dev_status=None):
        dev, n = ctx_len.device, ctx_len.shape[0]
        a = PagePlanArgs()
        a.ctx_len = _dense(ctx_len, "ctx_len", torch.int32, (n,))
        a.new_len = _dense(new_len, "new_len", torch.int32, (n,), dev)
        if table.dim() != 2:
            raise ValueError("table must be [sequences, columns]")
        a.table = _dense(table, "table", torch.int32, (n, table.shape[1]), dev)
        a.free_pages = _dense(free_pages, "free_pages", torch.int32, (free_pages.numel(),), dev)
        a.n_seq, a.page_size, a.table_cols = n, _int(page_size, "page_size"), table.shape[1]
        a.n_free, a.max_rows = free_pages.numel(), _int(max_rows, "max_rows")
        self.table = table
        self.row_start = torch.empty(n + 1, dtype=torch.int32, device=dev)
        self.kv_len = torch.empty(n, dtype=torch.int32, device=dev)
        self.n_taken = torch.empty(1, dtype=torch.int32, device=dev)
        self.seq_of_row = torch.empty(max_rows, dtype=torch.int32, device=dev)
        self.pos = torch.empty(max_rows, dtype=torch.int64, device=dev)
        self.slot = torch.empty(max_rows, dtype=torch.int64, device=dev)
        mine = (self.row_start, self.kv_len, self.n_taken, self.seq_of_row, self.pos, self.slot)
        a.row_start, a.kv_len, a.n_taken, a.seq_of_row, a.pos, a.slot = (t.data_ptr() for t in mine)
        a.dev_status = None if dev_status is None else _dense(dev_status, "dev_status", torch.int32, (1,), dev)
        self._bind(_page_plan, a, dev, mine, (ctx_len, new_len, table, free_pages, dev_status))

    def __call__(self):
        self._run()
        return self


def page_plan(ctx_len, new_len, table, free_pages, page_size: int, max_rows: int, dev_status=None):
    """Page table entries and slot map of new tokens (see PagePlan); returns the PagePlan after
    running it."""
    return PagePlan(ctx_len, new_len, table, free_pages, page_size, max_rows, dev_status)()


# ------------------------------------------------------------------ rotary axes
class RopeAxes(_Prepared):
    """A prepared csa2_rope_axes call: x [T, heads, dim] (bf16, fp16 or fp32; rows and heads may be
    strided) turned by pos [axes, T] int64 ([T] for one axis).  `sections` gives each axis its number
    of consecutive pairs, `axis_of_pair` any other assignment; without either, one axis.  `pairing`:
    "half" pairs dim i with i + rot_dim / 2, "adjacent" 2i with 2i + 1.  `inverse` turns back, which is
    the gradient.  `out` may be x itself.  A prepared call builds no autograd graph: an x whose gradient
    torch would track is refused (rope_axes without `out` takes it)."""
    _name = "csa2_rope_axes"

    def __init__(self, x, pos, sections=None, axis_of_pair=None, theta: float = 10000.0, rot_dim=None,
                 rot_first: int = 0, pairing: str = "half", inverse: bool = False, out=None):
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("x requires a gradient, which a prepared call or one with `out` does not record: call rope_axes "
                             "without `out`, or under torch.no_grad()")
        dev = x.device
        a = RopeAxesArgs()
        a.x, a.x_row, a.x_head = _heads(x, "x")
        T, H, D = x.shape
        if pos.dim() == 1:
            pos = pos[None]
        a.pos = _dense(pos, "pos", torch.int64, (pos.shape[0], T), dev)
        R = D - rot_first if rot_dim is None else int(rot_dim)
        if not 0 < R <= 2 * ROPE_AXES_MAX_PAIRS or R % 2:
            raise ValueError(f"rot_dim must be an even number of at most {2 * ROPE_AXES_MAX_PAIRS}")
        if sections is not None and axis_of_pair is not None:
            raise ValueError("give sections or axis_of_pair, not both")
        if sections is not None:
            axis_of_pair = [i for i, n in enumerate(sections) for _ in range(n)]
        if axis_of_pair is None:
            axis_of_pair = [0] * (R // 2)
        if len(axis_of_pair) != R // 2 or any(not 0 <= i < pos.shape[0] for i in axis_of_pair):
            raise ValueError("every pair of rot_dim / 2 needs one of pos's axes")
        if pairing not in ("half", "adjacent"):
            raise ValueError('pairing is "half" or "adjacent"')
        if out is None:
            out = torch.empty((T, H, D), dtype=x.dtype, device=dev)
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have x's shape and type")
        if any(n > 1 and t == 0 for n, t in zip(out.shape, out.stride())):
            raise ValueError("out must not be a broadcast tensor")
        self.out = out
        a.out, a.out_row, a.out_head = _heads(out, "out", dev)
        a.n_tokens, a.n_heads, a.head_dim, a.dtype, a.n_axes = T, H, D, _TYPES[x.dtype], pos.shape[0]
        a.rot_first, a.rot_dim, a.half_pairs, a.inverse = _int(rot_first, "rot_first"), R, pairing == "half", bool(inverse)
        a.theta = float(theta)
        a.axis_of_pair[:R // 2] = list(axis_of_pair)
        self._bind(_rope_axes, a, dev, (out,), (x, pos))

    def __call__(self):
        self._run()
        return self.out


class _Turn(torch.autograd.Function):
    """rope_axes where x's gradient is tracked: the gradient is turned back."""

    @staticmethod
    def forward(ctx, x, pos, how, inverse):
        ctx.save_for_backward(pos)
        ctx.how, ctx.inverse = how, inverse
        return RopeAxes(x, pos, *how, inverse)()

    @staticmethod
    def backward(ctx, grad):
        grad = grad.contiguous()  # a sum's gradient is a broadcast tensor
        if grad.data_ptr() % 16:
            grad = grad.clone()
        return rope_axes(grad, ctx.saved_tensors[0], *ctx.how, not ctx.inverse), None, None, None


def rope_axes(x, pos, sections=None, axis_of_pair=None, theta: float = 10000.0, rot_dim=None, rot_first: int = 0,
              pairing: str = "half", inverse: bool = False, out=None):
    """x with its rotary dims turned by positions of several axes (see RopeAxes).  Differentiable in x
    unless `out` is given."""
    if out is None and x.requires_grad and torch.is_grad_enabled():
        sections, axis_of_pair = (None if v is None else tuple(v) for v in (sections, axis_of_pair))  # for both passes
        return _Turn.apply(x, pos, (sections, axis_of_pair, theta, rot_dim, rot_first, pairing), bool(inverse))
    return RopeAxes(x, pos, sections, axis_of_pair, theta, rot_dim, rot_first, pairing, inverse, out)()


# ------------------------------------------------------------------ cache
class PageCache(NamedTuple):
    """Codes [pages, kv heads, page size, dim] uint8 (E4M3) of keys and values, and their scales
    [pages, kv heads] fp32: value = code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @staticmethod
    def empty(n_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> "PageCache":
        codes = [torch.empty((n_pages, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device) for _ in "kv"]
        scales = [torch.empty((n_pages, kv_heads), dtype=torch.float32, device=device) for _ in "kv"]
        return PageCache(*codes, *scales)


def _cache_fields(a, cache, device):
    if cache.k.dim() != 4:
        raise ValueError("cache codes must be [pages, kv heads, page size, dim]")
    n, h, p, d = cache.k.shape
    a.k_codes = _dense(cache.k, "cache.k", torch.uint8, (n, h, p, d), device)
    a.v_codes = _dense(cache.v, "cache.v", torch.uint8, (n, h, p, d), device)
    a.k_scale = _dense(cache.k_scale, "cache.k_scale", torch.float32, (n, h), device)
    a.v_scale = _dense(cache.v_scale, "cache.v_scale", torch.float32, (n, h), device)
    a.n_pages, a.kv_heads, a.page_size, a.head_dim = n, h, p, d


def _seq_fields(a, row_start, kv_len, table, device):
    n = kv_len.shape[0]
    if table.dim() != 2:
        raise ValueError("table must be [sequences, columns]")
    a.row_start = _dense(row_start, "row_start", torch.int32, (n + 1,), device)
    a.kv_len = _dense(kv_len, "kv_len", torch.int32, (n,), device)
    a.table = _dense(table, "table", torch.int32, (n, table.shape[1]), device)
    a.n_seq, a.table_cols = n, table.shape[1]


class PageWriter(_Prepared):
    """A prepared csa2_write_pages call: rows k and v [T, kv heads, dim] (bf16, fp16 or fp32; rows and
    heads may be strided) of the plan's new tokens into `cache`."""
    _name = "csa2_write_pages"

    def __init__(self, cache: PageCache, k, v, row_start, kv_len, seq_of_row, table, dev_status=None):
        dev = cache.k.device
        a = WritePagesArgs()
        _cache_fields(a, cache, dev)
        _seq_fields(a, row_start, kv_len, table, dev)
        a.k, a.k_row, a.k_head = _heads(k, "k", dev)
        a.v, a.v_row, a.v_head = _heads(v, "v", dev)
        if k.dtype != v.dtype or k.shape != v.shape or tuple(k.shape[1:]) != (a.kv_heads, a.head_dim):
            raise ValueError("k and v must be [rows, kv heads, dim] of the cache's heads and of one type")
        a.seq_of_row = _dense(seq_of_row, "seq_of_row", torch.int32, (k.shape[0],), dev)
        a.n_rows, a.dtype = k.shape[0], _TYPES[k.dtype]
        a.dev_status = None if dev_status is None else _dense(dev_status, "dev_status", torch.int32, (1,), dev)
        self._bind(_write_pages, a, dev, (), (cache, k, v, row_start, kv_len, seq_of_row, table, dev_status))

    def __call__(self):
        self._run()


def write_pages(cache: PageCache, k, v, row_start, kv_len, seq_of_row, table, dev_status=None) -> None:
    """Appends key and value rows to a paged 8-bit cache (see PageWriter)."""
    PageWriter(cache, k, v, row_start, kv_len, seq_of_row, table, dev_status)()


# ------------------------------------------------------------------ attention
class PagedAttn(_Prepared):
    """A prepared csa2_paged_attn call: q [T, heads, dim] (bf16 or fp16; rows and heads may be strided)
    over `cache`, out [T, heads, dim] in q's type (or out_dtype)."""
    _name = "csa2_paged_attn"

    def __init__(self, q, cache: PageCache, row_start, kv_len, table, softmax_scale: float, window: int = 0, sink=None,
                 out=None, out_dtype=None, dev_status=None):
        dev = q.device
        a = PagedAttnArgs()
        _cache_fields(a, cache, dev)
        _seq_fields(a, row_start, kv_len, table, dev)
        a.q, a.q_row, a.q_head = _heads(q, "q", dev)
        if q.dtype == torch.float32 or q.shape[2] != a.head_dim or q.shape[1] % max(a.kv_heads, 1):
            raise ValueError("q must be bf16 or fp16 [rows, heads, dim] with the cache's dim and a multiple of its heads")
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=dev)
        if out.dtype not in _TYPES or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must be bfloat16, float16 or float32")
        self.out = out
        a.out = _dense(out, "out", out.dtype, q.shape, dev)
        a.sink = None if sink is None else _dense(sink, "sink", torch.float32, (q.shape[1],), dev)
        a.n_rows, a.heads, a.q_dtype, a.out_dtype = q.shape[0], q.shape[1], _TYPES[q.dtype], _TYPES[out.dtype]
        a.softmax_scale, a.window = float(softmax_scale), _int(window, "window")
        a.dev_status = None if dev_status is None else _dense(dev_status, "dev_status", torch.int32, (1,), dev)
        self._wsp, a.workspace_bytes = _ws(int(_paged_attn_ws(C.byref(a))), dev)
        a.workspace = None if self._wsp is None else self._wsp.data_ptr()
        mine = (out,) if self._wsp is None else (out, self._wsp)
        self._bind(_paged_attn, a, dev, mine, (q, cache, row_start, kv_len, table, sink, dev_status))

    def __call__(self):
        self._run()
        return self.out


def paged_attn(q, cache: PageCache, row_start, kv_len, table, softmax_scale: float, window: int = 0, sink=None, out=None,
               out_dtype=None, dev_status=None):
    """Attention of the new tokens' queries over a paged 8-bit cache (see PagedAttn)."""
    return PagedAttn(q, cache, row_start, kv_len, table, softmax_scale, window, sink, out, out_dtype, dev_status)()


def selftest_paged_waits(call: PagedAttn, tries: int) -> None:
    """Runs a prepared call (with a dev_status) whose waits give up after `tries` tries
    (csa2_selftest_paged_waits): its status then reads ETIMEOUT and its output holds anything."""
    with torch.cuda.device(call._device):
        _check(_paged_waits(call._ref, int(tries), _raw_stream(call._index)), "csa2_selftest_paged_waits")
