"""More of the paged cache's entry points on a machine without a GPU: what is refused before anything is launched."""
import ctypes as C

import pytest
import torch

S = pytest.importorskip("sparse_attention_csa2_gb300")
from sparse_attention_csa2_gb300 import paged as P  # noqa: E402
from test_paged_host import ATTN, _fill  # noqa: E402


@pytest.mark.parametrize("tries,status,bad", [(-1, 1, {}), ((1 << 20) + 1, 1, {}), (5, 1, dict(dev_status=None)), (5, 1, dict(window=-1)),
                                              (5, 5, dict(workspace=None))])
def test_the_waits_self_test_refuses(tries, status, bad):
    a = _fill(P.PagedAttnArgs, **{**ATTN, "dev_status": 1 << 20, **bad})
    assert P._paged_waits(C.byref(a), tries, None) == status
    assert P._paged_waits(None, tries, None) == 1


def test_shapes_that_the_struct_would_cut_are_refused():
    x = torch.empty((1, 1, 64), dtype=torch.bfloat16).expand(2 ** 32 + 4, 1, 64)
    with pytest.raises(ValueError, match="2\\^31"):
        P._heads(x, "x")
    with pytest.raises(ValueError, match="2\\^31"):
        P._dense(torch.empty((0, 2 ** 31), dtype=torch.int32), "table", torch.int32, (0, 2 ** 31))
    with pytest.raises(ValueError, match="CUDA"):
        P._heads(torch.empty((1, 1, 64), dtype=torch.bfloat16).expand(2 ** 31 - 1, 1, 64), "x")
