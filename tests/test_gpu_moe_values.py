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


@pytest.mark.parametrize("form", ["few", "many"])
@pytest.mark.parametrize("w_codes", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_h_itself_to_its_bits(w_codes, T, form):
    """One column of x and one weight a row, all 1: an output is h of that row, which has no sums to hide in."""
    D = F = 256
    rng = np.random.default_rng(34)
    up, down = np.zeros((1, 2 * F, D), np.float32), np.zeros((1, D, F), np.float32)
    up[0, :, 0] = np.exp2(rng.integers(-3, 3, 2 * F)) * rng.integers(8, 16, 2 * F) / 8 * rng.choice([-1, 1], 2 * F)  # E4M3's bits
    down[0, np.arange(D), rng.permutation(F)] = 1
    if w_codes:
        code = lambda m: torch.from_numpy(m).to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
        w = S.ExpertWeights(code(up), code(down), torch.ones((1, 2 * F), device="cuda"), torch.ones((1, D), device="cuda"))
    else:
        w = S.ExpertWeights(*(torch.from_numpy(m).bfloat16().cuda() for m in (up, down)))
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    got = S.moe_experts(x, torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda"), w, out_dtype=torch.float32, form=form)
    g, u = up[0, :F, 0].astype(np.float64), up[0, F:, 0].astype(np.float64)
    want = (g / (1 + np.exp(-g)) * u)[down[0].argmax(1)]
    # the exponential is good to 2^-22, a sum, a quotient and a product round by 2^-24 each; then the parts: three bf16 are
    # fp32, two fp16 leave 2^-22, two bf16 2^-17 (each takes 8 bits and a sign of what the last one left)
    eps = 2.0 ** -22 + 3 * 2.0 ** -24 + (2.0 ** -17 if form == "many" else 2.0 ** -22 if w_codes else 0)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= eps * np.abs(want))
