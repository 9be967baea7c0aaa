"""The paged cache's entry points on a machine without a GPU: refusals of both the C ABI and the Python
calls before anything is launched, workspace sizes, and the oracle's own pins."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle.paged as OP

S = pytest.importorskip("sparse_attention_csa2_gb300")
from sparse_attention_csa2_gb300 import paged as P  # noqa: E402

A = 1 << 20  # an aligned stand-in address: every refused case fails before any use


def _fill(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


PLAN = dict(ctx_len=A, new_len=A, n_seq=4, page_size=16, table=A, table_cols=8, free_pages=A, n_free=9, max_rows=4,
            row_start=A, kv_len=A, seq_of_row=A, pos=A, slot=A, n_taken=A)
ROPE = dict(n_tokens=4, n_heads=2, head_dim=64, dtype=P.T_BF16, x=A, x_row=128, x_head=64, out=2 * A, out_row=128,
            out_head=64, pos=A, n_axes=1, rot_first=0, rot_dim=64, half_pairs=1, inverse=0, theta=1e4)
WRITE = dict(n_rows=4, n_seq=2, kv_heads=2, head_dim=64, page_size=16, n_pages=9, table_cols=4, dtype=P.T_BF16, k=A,
             k_row=128, k_head=64, v=A, v_row=128, v_head=64, row_start=A, kv_len=A, seq_of_row=A, table=A, k_codes=A,
             v_codes=A, k_scale=A, v_scale=A)
ATTN = dict(n_rows=4, n_seq=2, heads=8, kv_heads=2, head_dim=64, page_size=16, n_pages=9, table_cols=4, q_dtype=P.T_BF16,
            out_dtype=P.T_BF16, q=A, q_row=512, q_head=64, row_start=A, kv_len=A, table=A, k_codes=A, v_codes=A, k_scale=A,
            v_scale=A, softmax_scale=0.1, window=0, out=A, workspace=A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("bad,status", [
    (dict(n_seq=-1), 1), (dict(max_rows=-1), 1), (dict(page_size=0), 1), (dict(page_size=65537), 1), (dict(table_cols=0), 1),
    (dict(n_seq=8193), 2), (dict(ctx_len=None), 1), (dict(table=None), 1), (dict(free_pages=None), 1),
    (dict(row_start=None), 1), (dict(n_taken=None), 1), (dict(slot=None), 1), (dict(pos=A + 8), 1), (dict(n_free=-1), 1)])
def test_page_plan_refusals(bad, status):
    assert P._page_plan(C.byref(_fill(P.PagePlanArgs, **{**PLAN, **bad})), None) == status
    assert P._page_plan(None, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(n_tokens=-1), 1), (dict(n_heads=0), 1), (dict(head_dim=60), 1), (dict(head_dim=4104), 2), (dict(dtype=3), 1),
    (dict(rot_dim=72), 1), (dict(rot_dim=8), 1), (dict(rot_first=4), 1), (dict(rot_first=8), 1), (dict(theta=0.0), 1),
    (dict(theta=float("nan")), 1), (dict(theta=float("inf")), 1), (dict(x=A + 2), 1), (dict(out=None), 1), (dict(pos=None), 1),
    (dict(x_row=129), 1), (dict(out_head=4), 1), (dict(out=A, out_row=256), 1), (dict(n_axes=0), 1), (dict(n_axes=17), 1),
    (dict(head_dim=512, rot_dim=272), 2)])
def test_rope_axes_refusals(bad, status):
    assert P._rope_axes(C.byref(_fill(P.RopeAxesArgs, **{**ROPE, **bad})), None) == status
    a = _fill(P.RopeAxesArgs, **ROPE)
    a.axis_of_pair[31] = 1  # an axis that pos does not have
    assert P._rope_axes(C.byref(a), None) == 1
    assert P._rope_axes(C.byref(_fill(P.RopeAxesArgs, **{**ROPE, "n_tokens": 0, "x": None})), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(n_rows=-1), 1), (dict(kv_heads=0), 1), (dict(kv_heads=65536), 2), (dict(head_dim=96), 2), (dict(page_size=24), 2),
    (dict(page_size=256), 2), (dict(dtype=-1), 1), (dict(k=None), 1), (dict(v=A + 4), 1), (dict(k_row=100), 1),
    (dict(v_head=63), 1), (dict(table=None), 1), (dict(k_scale=None), 1), (dict(v_codes=A + 8), 1), (dict(seq_of_row=None), 1)])
def test_write_pages_refusals(bad, status):
    assert P._write_pages(C.byref(_fill(P.WritePagesArgs, **{**WRITE, **bad})), None) == status
    assert P._write_pages(C.byref(_fill(P.WritePagesArgs, **{**WRITE, "n_rows": 0, "k": None})), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(n_rows=-1), 1), (dict(heads=7), 1), (dict(heads=0), 1), (dict(head_dim=256), 2), (dict(page_size=8), 2),
    (dict(q_dtype=P.T_F32), 1), (dict(out_dtype=5), 1), (dict(window=-1), 1), (dict(softmax_scale=float("nan")), 1),
    (dict(q=None), 1), (dict(q=A + 8), 1), (dict(q_row=509), 1), (dict(out=A + 4), 1), (dict(k_scale=None), 1),
    (dict(workspace=None), 5), (dict(workspace_bytes=100), 5), (dict(n_rows=1 << 30), 2), (dict(table_cols=1 << 28), 2)])
def test_paged_attn_refusals(bad, status):
    assert P._paged_attn(C.byref(_fill(P.PagedAttnArgs, **{**ATTN, **bad})), None) == status
    assert P._paged_attn_ws(None) == 0
    assert P._paged_attn(C.byref(_fill(P.PagedAttnArgs, **{**ATTN, "n_rows": 0, "q": None})), None) == 0


def test_python_calls_refuse_cpu_tensors_and_wrong_shapes():
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        S.page_plan(i32(3), i32(3), i32(3, 4), i32(5), 16, 3)
    with pytest.raises(ValueError):
        S.rope_axes(torch.zeros(4, 2, 64), torch.zeros((1, 4), dtype=torch.int64))
    with pytest.raises(ValueError):
        S.rope_axes(torch.zeros(4, 2, 64, dtype=torch.float64), torch.zeros((1, 4), dtype=torch.int64))
    cache = S.PageCache.empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        S.write_pages(cache, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), i32(4), i32(3), i32(3), i32(3, 4))
    with pytest.raises(ValueError):
        S.paged_attn(torch.zeros(3, 4, 64, dtype=torch.bfloat16), cache, i32(4), i32(3), i32(3, 4), 0.125)


# ------------------------------------------------------------------ the oracle's pins
@pytest.mark.parametrize("v", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 16])
def test_python_calls_refuse_numbers_that_the_struct_would_cut(v):
    with pytest.raises(ValueError):
        P._int(v, "window")
    assert P._int(2 ** 31 - 1, "window") == 2 ** 31 - 1


def test_oracle_e4m3_rounding_matches_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * np.exp2(rng.integers(-12, 9, 4000)), OP.e4m3_values()[:127],
                        (OP.e4m3_values()[:126] + OP.e4m3_values()[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OP.e4m3_codes(x.astype(np.float64)), want)
    vals = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OP.e4m3_values(), vals, equal_nan=True)


def test_oracle_attention_matches_dense_softmax():
    rng = np.random.default_rng(1)
    k, v = (OP.e4m3_codes(rng.standard_normal((3, 1, 16, 8)) * 70) for _ in "kv")
    ks, vs = np.full((3, 1), 2.0 ** -6), np.full((3, 1), 2.0 ** -7)
    q = rng.standard_normal((5, 2, 8))
    out, _, _ = OP.paged_attn(q, k, v, ks, vs, [0, 5], [37], np.array([[2, 0, 1]]), 0.3)
    val = OP.e4m3_values()
    kk = np.concatenate([val[k[g, 0]] * ks[g, 0] for g in (2, 0, 1)])[:37]
    vv = np.concatenate([val[v[g, 0]] * vs[g, 0] for g in (2, 0, 1)])[:37]
    z = np.einsum("thd,jd->thj", q, kk) * 0.3
    mask = np.arange(37)[None] > np.arange(32, 37)[:, None]
    z = np.where(mask[:, None], -np.inf, z)
    w = torch.softmax(torch.from_numpy(z), -1).numpy()
    assert np.allclose(out, w @ vv, atol=1e-12)


def test_oracle_plan_and_rotation_small_cases():
    table, rs, kv, seq, pos, slot, taken, ok = OP.page_plan(np.array([3, 0]), np.array([2, 1]), np.array([[7, -1], [-1, -1]]),
                                                            np.array([5, 9, 1]), 4, 4)
    assert table.tolist() == [[7, 5], [9, -1]] and rs.tolist() == [0, 2, 3] and kv.tolist() == [5, 1]
    assert seq.tolist() == [0, 0, 1, -1] and pos.tolist() == [3, 4, 0, -1] and slot.tolist() == [31, 20, 36, -1]
    assert taken == 2 and ok
    x = np.array([[[1.0, 0.0, 0.0, 2.0]]])
    y = OP.rope_axes(x, np.array([[3], [5]]), [0, 1], 100.0, half=False)
    assert np.allclose(y[0, 0], [np.cos(3), np.sin(3), -2 * np.sin(0.5), 2 * np.cos(0.5)])
