"""Paged attention over many sequences: every form's way to find its place on the line of work, with
several sequences per thread and where the choice of form changes."""
import numpy as np
import pytest
import torch

import oracle.paged as OP
from paged_bounds import attend
from paged_testlib import cuda, make, values

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _run(c, G, dtype="bf16", window=0, seed=0):
    D, rng = c["D"], np.random.default_rng(seed)
    q, qd = values((c["rows"], c["H"] * G, D), rng, dtype)
    cache = S.PageCache(*(cuda(c[k]) for k in ("k", "v", "ks", "vs")))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), D ** -0.5, window=window,
                       out_dtype=torch.float32, dev_status=status).double().cpu().numpy()
    ref, tol = attend(qd, c, D ** -0.5, window, None, 2.0 ** -22)
    assert S.read_device_status(status) == S.OK
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("n", [31, 32, 33, 128, 129, 400, 1100])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 2), (64, 16), (128, 16), (128, 32)])
def test_a_decode_step_of_many_sequences(n, D, G):
    rng = np.random.default_rng(n)
    kv = rng.integers(0, 150, n)  # some rows see no token at all
    kv[rng.integers(n)] = 900
    _run(make([1] * n, kv, 16, 1, D, seed=n), G)


@pytest.mark.parametrize("n", [33, 321, 513, 1100])
@pytest.mark.parametrize("D,G,most", [(64, 4, 4), (128, 4, 4), (128, 4, 8), (64, 4, 30), (128, 4, 30)])
def test_drafts_and_prompts_of_many_sequences(n, D, G, most):
    """Ragged, every fourth without a row."""
    rng = np.random.default_rng(n + most)
    new = rng.integers(most // 2 + 1, most * 3 // 2 + 2, n)
    new[rng.random(n) < 0.25] = 0
    _run(make(new, new + rng.integers(0, 60, n), 16, 1, D, seed=n), G, window=0 if n % 2 else 40)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("n", [9000, 16384, 16385])
def test_prompts_of_thousands_of_sequences(n, D, dtype):
    """Tiles of 256 up to 16,384 sequences, small tiles beyond."""
    rng = np.random.default_rng(n)
    new = rng.integers(2, 4, n)
    _run(make(new, new + rng.integers(0, 20, n), 16, 1, D, seed=n), 16, dtype)


def test_the_plan_reads_only_the_page_that_new_rows_join():
    """A negative entry there is reported, and its rows have no slot; entries of full pages are not read."""
    for at, ctx, bad in ((1, 20, True), (0, 20, False), (1, 32, False)):
        table = np.array([[4, 5, -1, -1]], np.int32)
        table[0, at] = -7
        t, status = cuda(table), torch.zeros(1, dtype=torch.int32, device="cuda")
        p = S.page_plan(cuda(np.array([ctx], np.int32)), cuda(np.array([14], np.int32)), t, cuda(np.array([8, 9], np.int32)), 16, 14,
                        dev_status=status)
        assert (S.read_device_status(status) == S.EDEVICE_INDEX) == bad
        join = 32 - ctx
        assert p.slot.tolist() == [-1 if bad else 5 * 16 + (ctx + i) % 16 for i in range(join)] + [8 * 16 + i for i in range(14 - join)]
        assert t.tolist() == [[*table[0, :2].tolist(), 8, -1]]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_writing_again_repeats_pages_with_a_nan(dtype):
    """A NaN among the rows that join a page of larger, smaller or NaN scale: the second call leaves what the first wrote."""
    c = make([3, 3, 3, 20], [40, 41, 42, 50], 16, 2, 64, seed=3)
    k, kd = values((c["rows"], 2, 64), np.random.default_rng(4), dtype)
    k[[1, 4, 7, 9], :, 5] = float("nan")
    kd = k.double().numpy()
    for b, s in enumerate((2.0 ** 8, 2.0 ** -20, np.nan, 2.0 ** 8)):
        for j in range((c["kv"][b] - c["new"][b]) // 16, -(-c["kv"][b] // 16)):
            c["ks"][c["table"][b, j]] = s
    c["vs"] = c["ks"].copy()
    cache = S.PageCache(*(cuda(c[x]) for x in ("k", "v", "ks", "vs")))
    seq = cuda(np.repeat(np.arange(4), c["new"]).astype(np.int32))
    args = (cache, k.cuda(), k.cuda(), cuda(c["row_start"]), cuda(c["kv"]), seq, cuda(c["table"]))
    S.write_pages(*args)
    once = [t.clone() for t in cache]
    rc, rs = OP.write_pages(c["k"], c["ks"], kd, c["row_start"], c["kv"], c["table"])
    assert np.array_equal(cache.k.cpu().numpy(), rc) and np.array_equal(cache.k_scale.cpu().numpy().astype(np.float64), rs, equal_nan=True)
    S.write_pages(*args)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(once, cache))


@pytest.mark.parametrize("D,G,new", [(64, 2, 1), (64, 16, 1), (128, 2, 1), (128, 16, 1), (128, 32, 1), (64, 2, 40), (128, 2, 40)])
def test_a_cache_without_pages_under_a_table_with_columns(D, G, new):
    """Tokens there are none of: rows of 0, nothing to report.  Tokens whose pages are not there: hidden and reported."""
    T = 3 * new
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, status = S.PageCache.empty(0, 2, 16, D), i32(0)
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    rows = i32(0, new, 2 * new, 3 * new)
    q = torch.randn((T, 2 * G, D), device="cuda").bfloat16()
    for kv, said in ((0, S.OK), (50, S.EDEVICE_INDEX)):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        S.paged_attn(q, cache, rows, i32(kv, kv, kv), table, 0.1, out=out, dev_status=status)
        assert S.read_device_status(status) == said and not bool(out.any())
    for t in (table, table[:, :0].contiguous()):
        status.zero_()
        seq = torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(new)
        S.write_pages(cache, q[:, :2], q[:, :2], rows, i32(new, new, new), seq, t, dev_status=status)
        assert S.read_device_status(status) == S.EDEVICE_INDEX


@pytest.mark.parametrize("D,G,new", [(64, 2, 1), (64, 8, 2), (128, 2, 1), (128, 8, 2), (128, 8, 4), (64, 2, 40), (128, 2, 40)])
def test_lengths_beyond_the_table(D, G, new):
    """Tokens beyond the table are not there; the rows' positions stay those of the length, so that each row sees all of
    the table, and under a window what of it is left."""
    c = make([new, new, new], [64, 64, 64], 16, 2, D, seed=7)
    c["table"] = np.ascontiguousarray(c["table"][:, :4])  # four pages each, all held
    rng = np.random.default_rng(8)
    q, qd = values((3 * new, 2 * G, D), rng, "bf16")
    cache = S.PageCache(*(cuda(c[x]) for x in ("k", "v", "ks", "vs")))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    over = np.array([0, 13, 1 << 20])
    for window in (0, 50):
        got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda((64 + over).astype(np.int32)), cuda(c["table"]), D ** -0.5,
                           window=window, out_dtype=torch.float32, dev_status=status).double().cpu().numpy()
        assert S.read_device_status(status) == S.OK
        for r in range(3 * new):
            p = 64 + over[r // new] - new + r % new  # its position
            seen, first = min(64, p + 1), max(0, p - window + 1) if window else 0
            if first >= seen:
                assert not got[r].any()
                continue
            one = dict(c, kv=np.array([seen], np.int32), row_start=np.array([0, 1], np.int32), table=c["table"][r // new][None])
            ref, tol = attend(qd[r:r + 1], one, D ** -0.5, seen - first, None, 2.0 ** -22)
            assert np.all(np.abs(got[r] - ref[0]) <= tol[0])
