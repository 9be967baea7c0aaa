"""The paged 8-bit cache on the GPU against its float64 oracle: page plan, rotary axes, page writer,
paged attention, and the four together over serving steps."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.paged as OP
from paged_testlib import TYPES, bound, cuda, make, values

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _same(a, b):
    return np.array_equal(a.cpu().numpy(), np.asarray(b).astype(a.cpu().numpy().dtype))


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("page", [1, 16, 48, 64])
@pytest.mark.parametrize("lens", ["decode", "prompts", "empty", "many", "one"])
def test_page_plan(page, lens):
    rng = np.random.default_rng(page)
    ctx, new = {"decode": (rng.integers(0, 200, 37), np.ones(37)), "prompts": (rng.integers(0, 90, 5), rng.integers(1, 3000, 5)),
                "empty": (np.array([0, 16, 0, 33, 0]), np.array([0, 0, 7, 0, 0])),
                "many": (rng.integers(0, 40, 1500), rng.integers(0, 4, 1500)), "one": (np.array([0]), np.array([1]))}[lens]
    ctx, new = ctx.astype(np.int32), new.astype(np.int32)
    cols = int((-(-(ctx + new) // page)).max()) + 2
    free = rng.permutation(100000).astype(np.int32)[: int((-(-(ctx + new) // page)).sum()) + 5]
    table = rng.integers(0, 1 << 20, (len(ctx), cols)).astype(np.int32)
    rows = int(new.sum()) + 9
    ref = OP.page_plan(ctx, new, table, free, page, rows)
    t, st = cuda(table), _status()
    p = S.page_plan(cuda(ctx), cuda(new), t, cuda(free), page, rows, dev_status=st)
    for again in range(2):  # a plan run again on its own table repeats it
        for got, want in zip((t, p.row_start, p.kv_len, p.seq_of_row, p.pos, p.slot), ref):
            assert _same(got, want)
        assert int(p.n_taken) == ref[6] and ref[7]
        p()
    assert S.read_device_status(st) == S.OK


def test_page_plan_short_of_pages_columns_and_rows():
    ctx, new = np.array([5, 0, 30], np.int32), np.array([20, 40, 10], np.int32)
    for free, cols, rows in ((np.arange(100, 102), 9, 70), (np.arange(100, 140), 2, 70), (np.arange(100, 140), 9, 33),
                             (np.zeros(0), 9, 70)):
        table, st = np.arange(3 * cols, dtype=np.int32).reshape(3, cols), _status()
        ref = OP.page_plan(ctx, new, table, free.astype(np.int32), 16, rows)
        t = cuda(table)
        p = S.page_plan(cuda(ctx), cuda(new), t, cuda(free.astype(np.int32)), 16, rows, dev_status=st)
        for got, want in zip((t, p.row_start, p.kv_len, p.seq_of_row, p.pos, p.slot), ref):
            assert _same(got, want)
        assert int(p.n_taken) == ref[6] and not ref[7]
        assert S.read_device_status(st) == S.EDEVICE_INDEX


def test_page_plan_without_sequences_and_with_negative_lengths():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    p = S.page_plan(z, z, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), z, 16, 5)
    assert p.row_start.tolist() == [0] and p.slot.tolist() == [-1] * 5 and int(p.n_taken) == 0
    p = S.page_plan(cuda(np.array([-3, 4], np.int32)), cuda(np.array([2, -9], np.int32)),
                    torch.zeros((2, 4), dtype=torch.int32, device="cuda"), cuda(np.arange(3, dtype=np.int32)), 16, 3)
    assert p.kv_len.tolist() == [2, 4] and p.seq_of_row.tolist() == [0, 0, -1]


def test_page_plan_lengths_beyond_an_int_stay_in_bounds_and_are_reported():
    """2^30 cached and as many new tokens are the most of a sequence; sums stay at the largest int."""
    top = 2 ** 31 - 1
    ctx, new = np.array([top, 7, 5, 3], np.int32), np.array([9, top, top, 1], np.int32)
    whole, st = np.arange(-100, 116, dtype=np.int32).reshape(54, 4), _status()
    t = cuda(whole)
    p = S.page_plan(cuda(ctx), cuda(new), t[25:29], cuda(np.array([500, 501, 502], np.int32)), 16, 60, dev_status=st)
    assert S.read_device_status(st) == S.EDEVICE_INDEX
    want = whole.copy()
    want[26, 1:], want[27, 1:], want[28, 1:] = [501, 502, -1], -1, whole[28, 1:]
    assert _same(t, want)
    assert p.row_start.tolist() == [0, 9, 9 + 2 ** 30 - 1, top, top]
    assert p.kv_len.tolist() == [2 ** 30 + 9, 2 ** 30 + 6, 2 ** 30 - 4, 3]
    assert p.seq_of_row.tolist() == [0] * 9 + [1] * 51
    assert p.pos.tolist() == list(range(2 ** 30, 2 ** 30 + 9)) + list(range(7, 58))
    pages = [whole[26, 0], 501, 502, -1]
    assert p.slot.tolist() == [-1] * 9 + [pages[i // 16] * 16 + i % 16 if pages[i // 16] >= 0 else -1 for i in range(7, 58)]


# ------------------------------------------------------------------ rotary axes
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,H,D,first,R,axes", [(1, 1, 16, 0, 16, 1), (5, 3, 64, 0, 64, 3), (33, 7, 192, 128, 64, 2),
                                                (130, 2, 128, 8, 96, 4), (3, 40, 256, 0, 256, 3)])
def test_rope_axes(dtype, half, T, H, D, first, R, axes):
    rng = np.random.default_rng(T + R)
    x, xv = values((T, H, D), rng, dtype, 2.0)
    pos = rng.integers(0, 1 << 20, (axes, T))
    pos[0, 0] = (1 << 31) - 1
    pos[-1, -1] = -77
    axis = [int(a) for a in rng.integers(0, axes, R // 2)]
    for inverse in (False, True):
        ref = OP.rope_axes(xv, pos, axis, 10000.0, first, half, inverse)
        got = S.rope_axes(x.cuda(), cuda(pos), axis_of_pair=axis, theta=10000.0, rot_dim=R, rot_first=first,
                          pairing="half" if half else "adjacent", inverse=inverse).double().cpu().numpy()
        # the angle: 2^-53 of its turns (2^31 * 0.16 of them at most, 2^-24.6 turns) and 2^-25 in its fp32
        # form, 2^-21.9 radians in all; sine, cosine, two products and a sum each 2^-23
        size = np.abs(xv).max(-1, keepdims=True)
        assert np.all(np.abs(got - ref) <= EPS[dtype] * np.abs(ref) + 2 * size * (2.0 ** -21.5 + 4 * 2.0 ** -23))


def test_rope_axes_sections_strides_and_in_place():
    rng = np.random.default_rng(3)
    qkv, qv = values((50, 12, 128), rng, "bf16")
    pos = rng.integers(0, 3000, (3, 50))
    axis = [0] * 16 + [1] * 24 + [2] * 24
    ref = OP.rope_axes(qv, pos, axis, 1e6)
    dev = qkv.cuda()
    q, k = dev[:, :8], dev[:, 8:10]
    want_q = S.rope_axes(q, cuda(pos), sections=(16, 24, 24), theta=1e6)  # out of place, strided input
    assert S.rope_axes(k, cuda(pos), sections=(16, 24, 24), theta=1e6, out=k) is k
    S.rope_axes(q, cuda(pos), sections=(16, 24, 24), theta=1e6, out=q)
    assert torch.equal(q, want_q) and torch.equal(dev[:, 10:].cpu(), qkv[:, 10:])
    got = dev[:, :10].double().cpu().numpy()
    assert np.all(np.abs(got - ref[:, :10]) <= 2.0 ** -8 * np.abs(ref[:, :10]) + 2.0 ** -18 * np.abs(qv).max())
    back = S.rope_axes(S.rope_axes(qkv.float().cuda(), cuda(pos), sections=(16, 24, 24)), cuda(pos), sections=(16, 24, 24),
                       inverse=True)
    assert torch.allclose(back.cpu(), qkv.float(), atol=1e-5)
    assert S.rope_axes(torch.zeros((0, 2, 64), device="cuda"), torch.zeros((1, 0), dtype=torch.int64, device="cuda")).shape[0] == 0


def test_rope_axes_inverse_is_the_gradient():
    """<R x, y> = <x, R^-1 y> for the formula's gradient, and central differences of sum(y * R x)."""
    rng = np.random.default_rng(4)
    x, xv = values((6, 2, 32), rng, "f32")
    y, yv = values((6, 2, 32), rng, "f32")
    pos = rng.integers(0, 5000, (2, 6))
    kw = dict(sections=(5, 11), theta=500.0)
    f = lambda t: S.rope_axes(t, cuda(pos), **kw)  # noqa: E731
    grad = S.rope_axes(y.cuda(), cuda(pos), inverse=True, **kw)
    size = np.abs(yv).max() * 2.0 ** -19
    assert np.all(np.abs(grad.double().cpu().numpy() - OP.rope_axes(yv, pos, [0] * 5 + [1] * 11, 500.0, inverse=True)) <= size)
    for _ in range(20):
        i = tuple(int(rng.integers(n)) for n in x.shape)
        d = torch.zeros_like(x)
        d[i] = 0.5  # the map is linear: a wide step is exact
        diff = ((f((x + d).cuda()).double() - f((x - d).cuda()).double()) * y.cuda().double()).sum().item()
        assert abs(diff - grad[i].item()) <= 64 * 2.0 ** -20 * np.abs(yv).max() * (1 + np.abs(xv).max())


# ------------------------------------------------------------------ writer
def _written(c, k, v, kd, vd, status=None):
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    seq = cuda(np.repeat(np.arange(len(c["new"])), c["new"]).astype(np.int32))
    S.write_pages(cache, k, v, cuda(c["row_start"]), cuda(c["kv"]), seq, cuda(c["table"]), dev_status=status)
    for codes, scale, got, gs, x in ((c["k"], c["ks"], cache.k, cache.k_scale, kd), (c["v"], c["vs"], cache.v, cache.v_scale, vd)):
        rc, rs = OP.write_pages(codes, scale, x, c["row_start"], c["kv"], c["table"])
        assert np.array_equal(got.cpu().numpy(), rc)  # the untouched slots and pages too
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), rs, equal_nan=True)
    return cache


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("batch", ["decode", "prompts", "mixed"])
def test_write_pages(dtype, D, page, batch):
    new, kv = {"decode": ([1] * 9, [1, 16, 17, 31, 100, 128, 129, 5, 64]), "prompts": ([300, 1, 77], [300, 40, 500]),
               "mixed": ([0, 2, 130, 0, 1, 16], [50, 2, 131, 0, 33, 16])}[batch]
    c = make(new, kv, page, 3, D, seed=D + page)
    rng = np.random.default_rng(7)
    lift = np.exp2(rng.integers(-6, 4, (c["rows"], 3, 1)))  # some pages' scales grow, some stay
    k, kd = values((c["rows"], 3, D), rng, dtype, lift)
    v, vd = values((c["rows"], 3, D), rng, dtype, lift[::-1])
    cache = _written(c, k.cuda(), v.cuda(), kd, vd)
    before = [t.clone() for t in cache]
    seq = cuda(np.repeat(np.arange(len(new)), new).astype(np.int32))
    S.write_pages(cache, k.cuda(), v.cuda(), cuda(c["row_start"]), cuda(c["kv"]), seq, cuda(c["table"]))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, cache))  # again: the same


def test_write_pages_odd_values():
    """Zero pages, the smallest and largest scales, ties at 448, infinities and NaN, and a page whose
    scale another writer chose."""
    c = make([16, 16, 16, 16, 16, 4, 4], [16, 16, 16, 16, 16, 8, 8], 16, 1, 64, seed=1)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((c["rows"], 1, 64)).astype(np.float32)
    x[0:16] = 0.0
    x[16:32] = 1e-38
    x[32:48] *= np.float32(3e38) / np.abs(x[32:48]).max()
    x[48, 0, :3] = [np.inf, -np.inf, 2.0]
    x[64, 0, 5] = np.nan
    x[49, 0, 0] = 448.0
    c["ks"][c["table"][5, 0]] = 0.013  # not a power of two, larger and smaller than needed
    c["ks"][c["table"][6, 0]] = 1e-5
    c["vs"][c["table"][6, 0]] = np.nan
    _written(c, torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), x.astype(np.float64), x.astype(np.float64))


def test_write_pages_strided_rows_bad_pages_and_rows_behind_the_last():
    c = make([3, 20], [40, 20], 16, 2, 64, seed=5)
    rng = np.random.default_rng(6)
    qkv, qd = values((c["rows"] + 4, 10, 64), rng, "bf16")
    dev = qkv.cuda()
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    seq = cuda(np.array([0] * 3 + [1] * 20 + [0, 1, -1, 9], np.int32))  # four rows behind the last sequence's
    S.write_pages(cache, dev[:, 6:8], dev[:, 8:10], cuda(c["row_start"]), cuda(c["kv"]), seq, cuda(c["table"]))
    rc, rs = OP.write_pages(c["k"], c["ks"], qd[:, 6:8], c["row_start"], c["kv"], c["table"])
    assert np.array_equal(cache.k.cpu().numpy(), rc)
    assert np.array_equal(cache.k_scale.cpu().numpy().astype(np.float64), rs, equal_nan=True)
    bad = c["table"].copy()
    bad[1, 0], bad[1, 1] = -1, 1 << 30
    st = _status()
    before = [t.clone() for t in cache]
    S.write_pages(cache, dev[:, 6:8], dev[:, 8:10], cuda(c["row_start"]), cuda(c["kv"]), seq, cuda(bad), dev_status=st)
    assert S.read_device_status(st) == S.EDEVICE_INDEX
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, cache))


# ------------------------------------------------------------------ attention
def _attend(c, heads, dtype, window=0, sink=False, out="f32", seed=0, spread=1.0, scale=None, table=None, status=None):
    rng = np.random.default_rng(seed)
    T, D = c["rows"], c["D"]
    q, qd = values((T, heads, D), rng, dtype, spread)
    scale = D ** -0.5 if scale is None else scale
    sk = rng.standard_normal(heads).astype(np.float32) if sink else None
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"] if table is None else table),
                       softmax_scale=scale, window=window, sink=None if sk is None else cuda(sk), out_dtype=TYPES[out],
                       dev_status=status)
    ref = OP.paged_attn(qd, c["k"], c["v"], c["ks"].astype(np.float64), c["vs"].astype(np.float64), c["row_start"], c["kv"],
                        c["table"], scale, window, sk)
    return got.double().cpu().numpy(), ref, bound(qd, c, ref, EPS[out] if out != "f32" else 2.0 ** -22)


BATCHES = {
    "one": ([1], [1]),
    "decode": ([1] * 7, [1, 15, 16, 17, 100, 333, 1000]),
    "long": ([1, 1], [9000, 1]),
    "drafts": ([4, 1, 3, 0, 5], [300, 50, 3, 77, 129]),
    "prompts": ([70, 33, 1], [70, 200, 90]),
    "shorter": ([6, 2, 3], [4, 0, 3]),  # fewer tokens than queries: their first rows see none
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 64), (64, 128), (128, 32)])
@pytest.mark.parametrize("batch", sorted(BATCHES))
@pytest.mark.parametrize("H,G", [(2, 1), (1, 3), (3, 8), (2, 16)])
def test_paged_attn(dtype, D, page, batch, H, G):
    c = make(*BATCHES[batch], page, H, D, seed=D + page + H)
    got, ref, tol = _attend(c, H * G, dtype)
    assert np.all(np.abs(got - ref[0]) <= tol)


@pytest.mark.parametrize("window", [1, 15, 16, 100])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("batch", ["decode", "drafts", "prompts", "shorter"])
@pytest.mark.parametrize("G", [4, 20])
def test_paged_attn_window_and_sink(window, sink, batch, G):
    c = make(*BATCHES[batch], 16, 2, 128, seed=window)
    for b in range(len(c["kv"])):  # pages wholly behind the window are gone
        first = max(0, int(c["kv"][b] - c["new"][b]) - window + 1) // 16
        c["table"][b, :first] = np.where(c["table"][b, :first] >= 0, c["table"][b, :first], -1)
    gone = c["table"].copy()
    for b in range(len(c["kv"])):
        gone[b, :max(0, int(c["kv"][b] - c["new"][b]) - window + 1) // 16] = -1
    st = _status()
    got, ref, tol = _attend(c, 2 * G, "bf16", window, sink, table=gone, status=st)
    assert np.all(np.abs(got - ref[0]) <= tol)
    assert S.read_device_status(st) == S.OK


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("batch", ["decode", "prompts"])
def test_paged_attn_output_types(out, batch):
    c = make(*BATCHES[batch], 32, 2, 64, seed=3)
    got, ref, tol = _attend(c, 6, "f16", out=out)
    assert np.all(np.abs(got - ref[0]) <= tol)


@pytest.mark.parametrize("batch", ["decode", "prompts"])
@pytest.mark.parametrize("what", ["sharp", "flat", "scales", "tiny_q", "huge_q"])
def test_paged_attn_ranges(batch, what):
    """Scores of hundreds, of nothing, page scales over 2^24, queries at the ends of bf16's range."""
    c = make(*BATCHES[batch], 16, 2, 128, seed=8, exps=(-18, 6) if what == "scales" else (-9, -4))
    spread, scale = {"sharp": (30.0, None), "flat": (1e-3, None), "scales": (0.02, None), "tiny_q": (1e-30, 1e30 / 12),
                     "huge_q": (1e30, 1e-30 / 12)}[what]
    got, ref, tol = _attend(c, 8, "bf16", spread=spread, scale=scale)
    assert np.all(np.abs(got - ref[0]) <= tol)


@pytest.mark.parametrize("batch", ["decode", "prompts"])
def test_paged_attn_nan_reaches_only_rows_that_see_it(batch):
    """A page marked NaN (in either scale) and a NaN query spoil the rows that they enter, no others."""
    c = make(*BATCHES[batch], 16, 2, 64, seed=9)
    b = len(c["kv"]) - 2
    g = c["table"][b, (c["kv"][b] - 1) // 16]
    first = (c["kv"][b] - 1) // 16 * 16
    clean, ref, tol = _attend(c, 4, "bf16")
    for which in ("ks", "vs"):
        d = dict(c, **{which: c[which].copy()})
        d[which][g, 1] = np.nan
        got, _, _ = _attend(d, 4, "bf16")
        for r in range(c["rows"]):
            s = np.searchsorted(c["row_start"], r, side="right") - 1
            sees = s == b and c["kv"][b] - c["row_start"][b + 1] + r >= first
            assert np.isnan(got[r, 2:]).all() if sees else np.array_equal(got[r, 2:], clean[r, 2:])
            assert np.array_equal(got[r, :2], clean[r, :2])


def test_paged_attn_bad_pages_and_lengths_are_hidden_and_reported():
    c = make([1, 40], [200, 100], 16, 2, 64, seed=10)
    bad, st = c["table"].copy(), _status()
    bad[0, 3], bad[1, 2] = 1 << 29, -5
    q, qd = values((41, 4, 64), np.random.default_rng(0), "bf16")
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(bad), 0.125, out_dtype=torch.float32,
                       dev_status=st).double().cpu().numpy()
    assert S.read_device_status(st) == S.EDEVICE_INDEX
    # the oracle: the same tokens with scores of -inf, by a key of -1e300 along a query dim that is 1
    val = OP.e4m3_values()
    for r in range(41):
        b = 0 if r < 1 else 1
        p = int(c["kv"][b] - c["row_start"][b + 1] + r)
        for h in range(4):
            ks, vs = [], []
            for t in range(p + 1):
                g = bad[b, t // 16]
                if 0 <= g < len(c["k"]):
                    ks.append(val[c["k"][g, h // 2, t % 16]] * float(c["ks"][g, h // 2]))
                    vs.append(val[c["v"][g, h // 2, t % 16]] * float(c["vs"][g, h // 2]))
            z = np.array(ks) @ qd[r, h] * 0.125
            w = np.exp(z - z.max())
            ref = w @ np.array(vs) / w.sum()
            assert np.all(np.abs(got[r, h] - ref) <= 2.0 ** -9 * (w @ np.abs(np.array(vs)) / w.sum()))
    # lengths beyond the table count as its end
    kv = c["kv"].copy()
    kv[0] = c["table"].shape[1] * 16 + 50
    S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda(kv), cuda(c["table"]), 0.125, dev_status=st)
    torch.cuda.synchronize()


@pytest.mark.parametrize("batch", ["decode", "drafts", "prompts"])
@pytest.mark.parametrize("D", [64, 128])
def test_paged_attn_lengths_beyond_every_table(batch, D):
    """A length at the largest int: the rows' places lie behind the table's tokens, all of which they see without a
    window, none with one."""
    c = make(*BATCHES[batch], 16, 2, D, seed=24)
    q, _ = values((c["rows"], 8, D), np.random.default_rng(5), "bf16")
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    long = torch.full((len(c["kv"]),), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), long, cuda(c["table"]), D ** -0.5, window=4000, out=out)
    assert not bool(got.any())
    table = cuda(np.zeros_like(c["table"]))  # page 0 all along
    full = torch.full_like(long, 16 * table.shape[1] + 10 ** 6)
    a = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), long, table, D ** -0.5)
    b = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), full, table, D ** -0.5)
    assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())


def test_paged_attn_leaves_rows_behind_the_last_and_takes_strided_queries():
    c = make([1, 2, 40], [50, 60, 70], 16, 2, 128, seed=11)
    T = c["rows"] + 5
    qkv, _ = values((T, 12, 128), np.random.default_rng(1), "bf16")
    dev = qkv.cuda()
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    args = (cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), 128 ** -0.5)
    out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    S.paged_attn(dev[:, 2:10], *args, out=out)
    dense = S.paged_attn(dev[:, 2:10].contiguous()[: c["rows"]], *args)
    assert torch.equal(out[: c["rows"]], dense) and bool((out[c["rows"]:] == 7.0).all())
    for _ in range(3):  # no atomics: bit for bit the same
        assert torch.equal(S.paged_attn(dev[:, 2:10], *args)[: c["rows"]], dense)


@pytest.mark.parametrize("batch", ["decode", "drafts", "prompts", "shorter"])
@pytest.mark.parametrize("G", [2, 12])
def test_paged_attn_scales_and_windows_at_their_ends(batch, G):
    """A softmax scale of 0 weighs all visible keys alike, a negative one turns the order; the largest window
    is none, also for sequences with fewer tokens than queries."""
    c = make(*BATCHES[batch], 16, 2, 128, seed=21)
    for scale in (0.0, -0.1):
        got, ref, tol = _attend(c, 2 * G, "bf16", scale=scale)
        assert np.all(np.abs(got - ref[0]) <= tol)
    plain, _, _ = _attend(c, 2 * G, "bf16")
    wide, _, _ = _attend(c, 2 * G, "bf16", window=2 ** 31 - 1)
    assert np.array_equal(plain, wide)


@pytest.mark.parametrize("batch", ["decode", "drafts", "prompts"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_paged_attn_query_that_is_not_finite_spoils_its_own_row(batch, D, bad):
    c = make(*BATCHES[batch], 32, 2, D, seed=22)
    T = c["rows"]
    q, _ = values((T, 8, D), np.random.default_rng(3), "bf16")
    cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
    args = (cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), D ** -0.5)
    clean = S.paged_attn(q.cuda(), *args)
    r, h = T // 2, 5
    q[r, h, 7] = bad
    got = S.paged_attn(q.cuda(), *args)
    assert bool(torch.isnan(got[r, h]).all())
    got[r, h] = clean[r, h]
    assert torch.equal(got, clean)


def test_paged_attn_between_other_kernels_of_the_framework():
    """Behind and before projections, whose kernels hold tensor memory and let the next kernel start early:
    every form of the attention in turn, on two streams at once."""
    cases = [make(*BATCHES[b], 64, 2, 128, seed=23) for b in ("decode", "drafts", "prompts")]
    rng = np.random.default_rng(4)
    x, _ = values((32, 512), rng, "bf16")
    w, _ = values((1024, 512), rng, "bf16")
    x, w = x.cuda(), w.cuda()
    calls = []
    for c in cases:
        q, _ = values((c["rows"], 8, 128), rng, "bf16")
        cache = S.PageCache(cuda(c["k"]), cuda(c["v"]), cuda(c["ks"]), cuda(c["vs"]))
        calls.append((q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), 128 ** -0.5))
    want_y = S.linear(x, w)
    want = [S.paged_attn(*a) for a in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(20):
                for a in calls:
                    got.append((S.linear(x, w), S.paged_attn(*a)))
    torch.cuda.synchronize()
    for i, (y, o) in enumerate(got):
        assert torch.equal(y, want_y) and torch.equal(o, want[i % 3])


@pytest.mark.parametrize("D,batch", [(64, "decode"), (128, "decode"), (128, "drafts"), (64, "prompts"), (128, "prompts")])
def test_pages_beyond_32_bit_offsets(D, batch):
    """The same tokens in the last pages of caches of more than 2^32 bytes and of their own pages only: codes, scales
    and outputs are equal bit for bit."""
    new, kv = BATCHES[batch]
    new = np.minimum(new, kv)
    c = make(new, kv, 64, 8, D, seed=25)
    n = len(c["k"])
    far = 2 ** 32 // (8 * 64 * D) + 7
    rng = np.random.default_rng(6)
    T = c["rows"]
    q, k, v = (values((T, h, D), rng, "bf16")[0].cuda() for h in (16, 8, 8))
    seq = cuda(np.repeat(np.arange(len(new)), new).astype(np.int32))
    row_start, kv_len = cuda(c["row_start"]), cuda(c["kv"])
    near, wide = S.PageCache(*(cuda(c[t]) for t in ("k", "v", "ks", "vs"))), S.PageCache.empty(far + n, 8, 64, D)
    outs = []
    for cache, shift in ((near, 0), (wide, far)):
        for t, key in zip(cache, ("k", "v", "ks", "vs")):
            t[shift:] = cuda(c[key])
        table = cuda(np.where(c["table"] < 0, -1, c["table"] + shift).astype(np.int32))
        S.write_pages(cache, k, v, row_start, kv_len, seq, table)
        outs.append(S.paged_attn(q, cache, row_start, kv_len, table, D ** -0.5))
    assert torch.equal(*outs) and bool(torch.isfinite(outs[0].float()).all())
    for x, y in zip(near, wide):
        assert torch.equal(x.view(torch.uint8), y[far:].contiguous().view(torch.uint8))


def test_rope_axes_beyond_32_bit_offsets():
    T, H, D = 70000, 256, 128  # 2.3e9 elements
    x = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-40:] = torch.randn((40, H, D), device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda")
    want = S.rope_axes(x[-40:].contiguous(), pos[-40:].contiguous())
    S.rope_axes(x, pos, out=x)
    assert torch.equal(x[-40:], want)


def test_paged_attn_of_a_cache_without_pages():
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    empty = S.PageCache.empty(0, 2, 16, 64)
    out = S.paged_attn(q, empty, rows, z, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), 0.125)
    assert not bool(out.any())
    one = S.PageCache.empty(1, 2, 16, 64)
    for t in one:
        t.view(torch.uint8).fill_(0x7F)
    out = S.paged_attn(q, one, rows, z, torch.zeros((3, 2), dtype=torch.int32, device="cuda"), 0.125)
    assert not bool(out.any())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,G", [(128, 4), (64, 9)])
def test_serving_steps(D, G):
    """Prompts, then decode steps with drafts: plan, rotation, write and attention each step, against the
    oracle's own cache; the plan's slots also place records of the framework's own cache."""
    H, page, n, theta = 2, 16, 4, 1e4
    rng = np.random.default_rng(12)
    pool = 64
    free = rng.permutation(pool).astype(np.int32)
    table = np.full((n, 12), -1, np.int32)
    cache = S.PageCache.empty(pool, H, page, D)
    for t in cache:
        t.view(torch.uint8).fill_(0x7F)
    kc, vc = (t.cpu().numpy() for t in cache[:2])
    ks, vs = (t.cpu().numpy().astype(np.float64) for t in cache[2:])
    dev_table, ctx, taken = cuda(table), np.zeros(n, np.int32), 0
    records = torch.zeros((pool * page, 512), dtype=torch.bfloat16, device="cuda")
    axis = [0] * (D // 8) + [1] * (D // 8) + [2] * (D // 4)
    for new in ([37, 1, 60, 16], [1, 1, 1, 1], [3, 0, 5, 1], [1, 2, 1, 1]):
        new = np.array(new, np.int32)
        T = int(new.sum())
        plan = S.page_plan(cuda(ctx), cuda(new), dev_table, cuda(free[taken:]), page, T)
        table, row_start, kv, seq, pos, slot, used, _ = OP.page_plan(ctx, new, table, free[taken:], page, T)
        q, qd = values((T, H * G, D), rng, "bf16")
        k, _ = values((T, H, D), rng, "bf16")
        v, vd = values((T, H, D), rng, "bf16")
        at = np.stack([pos, pos // 7, pos % 7])
        spans = (D // 8, D // 8, D // 4)
        qr = S.rope_axes(q.cuda(), cuda(at), sections=spans, theta=theta)
        kr = S.rope_axes(k.cuda(), cuda(at), sections=spans, theta=theta)
        ref_q = OP.rope_axes(qd, at, axis, theta)
        assert np.all(np.abs(qr.double().cpu().numpy() - ref_q) <= 2.0 ** -8 * np.abs(ref_q) + 2.0 ** -17)
        S.write_pages(cache, kr, v.cuda(), plan.row_start, plan.kv_len, plan.seq_of_row, dev_table)
        out = S.paged_attn(qr, cache, plan.row_start, plan.kv_len, dev_table, D ** -0.5, out_dtype=torch.float32)
        kc, ks = OP.write_pages(kc, ks, kr.double().cpu().numpy(), row_start, kv, table)
        vc, vs = OP.write_pages(vc, vs, vd, row_start, kv, table)
        assert np.array_equal(cache.k.cpu().numpy(), kc) and np.array_equal(cache.v.cpu().numpy(), vc)
        qq = qr.double().cpu().numpy()
        ref = OP.paged_attn(qq, kc, vc, ks, vs, row_start, kv, table, D ** -0.5)
        tol = bound(qq, {"vs": vs, "kv": kv}, ref, 2.0 ** -22)
        assert np.all(np.abs(out.double().cpu().numpy() - ref[0]) <= tol)
        x = torch.randn((T, 512), device="cuda")
        S.write_records(x, plan.slot, records, None, S.BF16)
        assert torch.equal(records[torch.from_numpy(slot).cuda()], x.to(torch.bfloat16))
        ctx, taken = kv.astype(np.int32), taken + used


def test_captured_step_follows_the_lengths():
    """A decode step of prepared calls captured into two CUDA graphs; both replayed in turn with other
    lengths and inputs give what the calls give one by one, on another stream too."""
    H, G, D, page, n = 2, 8, 128, 16, 5
    c = make([1] * n, [40, 90, 17, 700, 3], page, H, D, seed=13)
    rng = np.random.default_rng(14)
    dev = {k: cuda(c[k]) for k in ("k", "v", "ks", "vs", "table")}
    cache = S.PageCache(dev["k"], dev["v"], dev["ks"], dev["vs"])
    spare = cuda(np.array([0, 1], np.int32))
    ctx, new = cuda(c["kv"] - 1), cuda(c["new"])
    q = torch.zeros((n, H * G, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((1, n), dtype=torch.int64, device="cuda")

    def step():
        plan = S.PagePlan(ctx, new, dev["table"], spare, page, n)
        calls = [plan, S.RopeAxes(q, pos), S.RopeAxes(k, pos)]
        calls.append(S.PageWriter(cache, calls[2].out, k, plan.row_start, plan.kv_len, plan.seq_of_row, dev["table"]))
        calls.append(S.PagedAttn(calls[1].out, cache, plan.row_start, plan.kv_len, dev["table"], D ** -0.5))
        return calls

    graphs = []
    for _ in range(2):
        calls = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for f in calls:
                f()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for f in calls:
                f()
        graphs.append((g, calls))
    for it in range(4):
        back = torch.from_numpy(rng.integers(0, 3, n).astype(np.int32)).cuda()
        ctx.copy_(cuda(c["kv"] - 1) - torch.minimum(back, cuda(c["kv"] - 1)))
        q.copy_(torch.randn(q.shape, device="cuda"))
        k.copy_(torch.randn(k.shape, device="cuda"))
        pos.copy_(ctx[None].long())
        saved = [t.clone() for t in cache]
        g, calls = graphs[it % 2]
        g.replay()
        got = calls[-1].out.clone()
        after = [t.clone() for t in cache]
        for t, s in zip(cache, saved):
            t.copy_(s)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            fresh = step()
            for f in fresh:
                f()
        torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(got, fresh[-1].out)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(after, cache))
