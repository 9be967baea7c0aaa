"""csa2_moe's results to the bits that its definition in csa2.h gives them, whatever the output's type and the form."""
import numpy as np
import pytest
import torch

from test_gpu_moe import layer, pick, rows

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("form", ["few", "many"])
@pytest.mark.parametrize("w_codes", [False, True])
@pytest.mark.parametrize("x_codes", [False, True])
@pytest.mark.parametrize("T", [3, 40])
def test_a_bf16_output_is_the_fp32_one_rounded(w_codes, x_codes, T, form):
    E, k, D, F = 4, 2, 272, 144
    w, _, _ = layer(E, 1, D, F, w_codes, 31)
    x, scale, _ = rows(T, D, x_codes, 32)
    ids, weights = (torch.from_numpy(v).cuda() for v in pick(T, E, k, 33))
    out = [S.moe_experts(x, ids, weights, w, n_shared=1, x_scale=scale, out_dtype=t, form=form) for t in (torch.float32, torch.bfloat16)]
    assert torch.equal(out[0].bfloat16(), out[1])
