"""Bounded waits of the paged attention made to run out, without faulting anything: with a few tries per wait,
while copies and products are under way, every form ends, says so and leaves the next call whole."""
import numpy as np
import pytest
import torch

from paged_testlib import cuda, make, values

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")

FORMS = {  # (new tokens, dim, heads of a group)
    "tiles of 8, dim 64": (1, 64, 8),
    "tiles of 8, dim 128": (1, 128, 8),
    "tiles of 16, dim 64": (1, 64, 16),
    "tiles of 16, dim 128": (1, 128, 16),
    "tiles of 32, dim 128": (1, 128, 32),
    "tiles of 256, dim 64": (40, 64, 4),
    "tiles of 256, dim 128": (40, 128, 4),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", list(FORMS))
def test_waits_that_run_out_end_the_call_and_are_reported(form, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    new, D, G = FORMS[form]
    c = make([new] * 9, [2500, 40, 700, 3000, 1, 129, 5000, 64, 1500], 64, 4, D, seed=31)
    q, _ = values((c["rows"], 4 * G, D), np.random.default_rng(1), dtype)
    cache = S.PageCache(*(cuda(c[k]) for k in ("k", "v", "ks", "vs")))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = S.PagedAttn(q.cuda(), cache, cuda(c["row_start"]), cuda(c["kv"]), cuda(c["table"]), D ** -0.5, dev_status=status)
    want = call().clone()
    assert S.read_device_status(status) == S.OK
    for tries in (0, 1, 1, 1, 2, 2, 3, 5, 1 << 20):
        status.zero_()
        S.selftest_paged_waits(call, tries)
        said = S.read_device_status(status)
        assert said == S.ETIMEOUT if tries == 0 else said in (S.OK, S.ETIMEOUT) if tries < 100 else said == S.OK
        if said == S.OK:
            assert torch.equal(call.out, want)
        status.zero_()
        assert torch.equal(call(), want) and S.read_device_status(status) == S.OK
