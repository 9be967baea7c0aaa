"""Paged attention over pages of very different V scales, every form, each row held to a bound of its own."""
import numpy as np
import pytest
import torch

import oracle.paged as OP
from paged_bounds import attend
from paged_testlib import cuda, make, values

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")

FORMS = {  # (new tokens, dim, heads of a group)
    "tiles of 8, dim 64": (1, 64, 8),
    "tiles of 8, dim 128": (1, 128, 8),
    "tiles of 16, dim 64": (5, 64, 3),
    "tiles of 16, dim 128": (4, 128, 4),
    "tiles of 32, dim 128": (4, 128, 8),
    "tiles of 256, dim 64": (40, 64, 4),
    "tiles of 256, dim 128": (75, 128, 4),
}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _check(c, form, dtype, q=None, window=0, sink=False, seed=0):
    _, D, G = FORMS[form]
    rng = np.random.default_rng(seed)
    if q is None:
        q, _ = values((c["rows"], c["H"] * G, D), rng, dtype)
    sk = rng.standard_normal(c["H"] * G).astype(np.float32) if sink else None
    cache = S.PageCache(*(cuda(c[k]) for k in ("k", "v", "ks", "vs")))
    got = S.paged_attn(q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), D ** -0.5, window=window,
                       sink=None if sk is None else cuda(sk), out_dtype=torch.float32).double().cpu().numpy()
    ref, tol = attend(q.double().numpy(), c, D ** -0.5, window, sk, 2.0 ** -22)
    assert np.all(np.abs(got - ref) <= tol)


def _batch(form, page=16, seed=0):
    new, D, _ = FORMS[form]
    kv = [max(k, new) for k in (1, 66, 200, 79, 1500, 333)]
    return make([new] * len(kv), kv, page, 2, D, seed=seed)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_large_page_that_some_rows_do_not_see(form, dtype):
    """The last page's V scale is 2^40 times the others': rows before it give what they give without it."""
    c = _batch(form, seed=1)
    for b, n in enumerate(c["kv"]):
        c["vs"][c["table"][b, (n - 1) // 16]] *= 2.0 ** 40
    _check(c, form, dtype)
    _check(c, form, dtype, window=30, sink=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_large_page_of_negligible_weight(form, at, dtype):
    """A page whose V scale is 2^40 times the others' and whose keys have softmax weights around 2^-70."""
    new, D, G = FORMS[form]
    c = _batch(form, seed=2)
    rng = np.random.default_rng(3)
    q = torch.from_numpy(1 + 0.1 * rng.random((c["rows"], 2 * G, D)).astype(np.float32)).to(dict(bf16=torch.bfloat16, f16=torch.float16)[dtype])
    size = 24 / D ** 0.5
    c["ks"][:] = np.where(np.isnan(c["ks"]), c["ks"], 2.0 ** -6)
    for b, n in enumerate(c["kv"]):
        pages = (n - 1) // 16 + 1
        far = {"first": 0, "middle": pages // 2, "last": pages - 1}[at]
        for j in range(pages):
            g, m = c["table"][b, j], min(16, n - 16 * j)
            sign = -1 if j == far and pages > 1 else 1
            c["k"][g, :, :m] = OP.e4m3_codes(64 * sign * size * (1 + 0.05 * rng.standard_normal((2, m, D))))
            if sign < 0:
                c["vs"][g] *= 2.0 ** 40
    _check(c, form, dtype, q)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("exps", [(-40, 10), (-100, -90), (-101, 1), (60, 71)])
def test_scales_over_the_range_of_the_writer(form, exps):
    c = _batch(form, seed=4)
    rng = np.random.default_rng(5)
    c["vs"] = np.where(np.isnan(c["vs"]), c["vs"], np.exp2(rng.integers(*exps, c["vs"].shape))).astype(np.float32)
    _check(c, form, "bf16", seed=6)
    _check(c, form, "bf16", sink=True, seed=7)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("small", [0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -126])
def test_scales_of_zero_and_below_the_normal_numbers(form, small):
    """Some pages, and all of them."""
    for some in (True, False):
        c = _batch(form, seed=8)
        rng = np.random.default_rng(9)
        c["vs"] = np.where(np.isnan(c["vs"]) | (rng.random(c["vs"].shape) < 0.5) & some, c["vs"], np.float32(small)).astype(np.float32)
        _check(c, form, "bf16")


@pytest.mark.parametrize("form", list(FORMS))
def test_scales_that_are_no_powers_of_two(form):
    c = _batch(form, seed=10)
    rng = np.random.default_rng(11)
    for s in ("ks", "vs"):
        c[s] = (c[s] * (0.5 + rng.random(c[s].shape))).astype(np.float32)
    _check(c, form, "bf16")
    _check(c, form, "f16", sink=True)
