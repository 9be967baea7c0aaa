"""csa2_moe's results to the bits that its definition in csa2.h gives them, whatever the output's type and the form."""
import numpy as np
import pytest
import torch

import oracle.step as OS
from test_gpu_moe import TYPES, layer, pick, rows

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


@pytest.mark.parametrize("form", ["few", "many"])
@pytest.mark.parametrize("w_codes", [False, True])
def test_sums_of_many_products_of_one_sign(w_codes, form):
    """8,192 columns: both forms hold 2^-15 of what is added.  (Sums that a tensor core cuts off towards 0 each time that it adds
    all err to one side; the up product's h is a sum itself, the down product's h have 15 bits and are exact.)"""
    n, T, F = 8192, 40, 128
    g = torch.Generator("cuda").manual_seed(35)
    rand = lambda *s: (1 + torch.rand(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731

    def weights(up, down):
        if not w_codes:
            return S.ExpertWeights(up, down), up.double(), down.double()
        codes = [m.to(torch.float8_e4m3fn) for m in (up, down)]
        w = S.ExpertWeights(*(c.view(torch.uint8) for c in codes), torch.ones(up.shape[:2], device="cuda"), torch.ones(down.shape[:2], device="cuda"))
        return w, *(c.double() for c in codes)

    def outputs(x, w):
        ids, ones = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda")
        return S.moe_experts(x, ids, ones, w, out_dtype=torch.float32, form=form).double()

    up, down = torch.zeros((1, 2 * F, n), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, n, F), dtype=torch.bfloat16, device="cuda")
    up[0, :F], up[0, F:, 0], x = rand(F, n), 1, rand(T, n)
    x[:, 0] = 1
    down[0, torch.arange(F), torch.arange(F)] = 1
    w, uv, _ = weights(up, down)
    want = x.double() @ uv[0, :F].T              # silu of thousands is the same, times 1
    assert torch.all((outputs(x, w)[:, :F] - want).abs() <= 2.0 ** -15 * want)

    up, down = torch.zeros((1, 2 * n, 64), dtype=torch.bfloat16, device="cuda"), rand(1, 64, n)
    up[0, :n, 0], up[0, n:, 1] = 96, 1
    x = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 1, rand(T)
    w, _, dv = weights(up, down)
    want = 96 * x[:, 1].double()[:, None] * dv[0].sum(1)
    assert torch.all((outputs(x, w) - want).abs() <= 2.0 ** -15 * want)


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("T", [1, 3, 9, 40])
def test_route_by_products_that_are_infinite(types, score, T):
    """An infinity in x makes every product infinite, by the weight's sign: scores of 1 (or infinity) and 0, of which the bias
    says the order.  Beside it rows as they are, and (fp32) rows whose products overflow."""
    D, E, k = 256, 48, 6
    g = torch.Generator().manual_seed(36)
    x = torch.randn(T, D, generator=g).to(TYPES[types[0]])
    w = torch.randn(E, D, generator=g).to(TYPES[types[1]])
    bias = torch.randperm(E, generator=g) / 100.0
    w[:, 7] = torch.where(torch.arange(E) % 3 == 0, 1.0, -1.0).to(w.dtype)  # 16 of 48 above
    x[0, 7] = float("inf")
    if T > 2:
        x[2, 7] = -float("inf")
    if T > 1 and types[0] == "f32":
        x[1] *= 2.0 ** 124                    # products are sums of some 2^128
    with_bias = score != "softmax"            # (with a bias, softmax's scores beside an infinite product are NaN)
    got = S.route_experts(x.cuda(), w.cuda(), k, bias=bias.cuda() if with_bias else None, score=score, normalize=False)
    # products beyond fp32's range as infinities, as they are compared
    z = x.double().numpy() @ w.double().numpy().T
    z = np.where(np.abs(z) >= 2.0 ** 128, np.sign(z) * np.inf, z)
    by = OS.score(z, score) + bias.double().numpy() if with_bias else z
    sure = [t for t in range(T) if not (types[0] == "f32" and t == 1)]   # (of a sum near 2^128 the order of addition decides)
    ids = np.stack([sorted(range(E), key=lambda e, r=r: (-r[e], e))[:k] for r in by])
    assert np.array_equal(got.ids.cpu().numpy()[sure], ids[sure])
    if with_bias:
        weights = np.take_along_axis(OS.score(z, score), ids, 1)[sure]
        mine = got.weights.double().cpu().numpy()[sure]
        inf = np.isinf(weights)
        # finite products as in test_gpu_moe.test_route: their rows are those without an infinity
        rest = [t for t in sure if t not in (0, 2)]
        dz = (D / 32 + 6) * 2.0 ** -24 * (np.abs(x.double().numpy()[rest]) @ np.abs(w.double().numpy()).T).max() if rest else 0.0
        assert np.array_equal(np.isinf(mine), inf) and np.all(np.abs(mine - weights)[~inf] <= (2 * dz + 2.0 ** -21) * weights[~inf])
    elif T > 3:
        assert got.weights[0].isnan().all() and got.weights[3].isfinite().all()


def test_route_weights_beside_a_nan():
    D, E = 64, 32
    x, w = torch.randn(5, D, device="cuda"), torch.randn(E, D, device="cuda")
    w[7], x[2] = float("nan"), float("nan")
    assert S.route_experts(x, w, 31).weights.isnan().all()       # of a softmax that holds one
    for score in ("sigmoid", "sqrtsoftplus"):
        got = S.route_experts(x, w, 31, score=score)
        assert got.weights[2].isnan().all() and got.weights[[0, 1, 3, 4]].isfinite().all()
        assert not (got.ids[[0, 1, 3, 4]] == 7).any()
        assert S.route_experts(x, w, 32, score=score, normalize=False).weights.isnan().sum(1).tolist() == [1, 1, 32, 1, 1]


@pytest.mark.parametrize("form", ["few", "many"])
@pytest.mark.parametrize("w_codes", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [4, 100])
def test_an_output_after_a_wait_that_ran_out_is_nan(w_codes, T, out, form):
    E, k, D, F = 4, 2, 1024, 512
    w, _, _ = layer(E, 1, D, F, w_codes, 37)
    x, _, _ = rows(T, D, False, 38)
    ids, weights = (torch.from_numpy(v).cuda() for v in pick(T, E, k, 39))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.zeros((T + 1, D + 8), dtype=out, device="cuda")
    call = S.MoEExperts(x, ids, weights, w, n_shared=1, dev_status=status, out=wide[:T, :D], form=form)
    want = call().clone()
    for tries in (0, 0, 1, 2, 3, 5, 8):
        status.zero_()
        S.selftest_moe_waits(call, tries)
        if S.read_device_status(status) == S.ETIMEOUT:
            assert call.out.isnan().all()
        else:
            assert tries and torch.equal(call.out, want)
        assert not wide[T].any() and not wide[:, D:].any()
        assert torch.equal(call(), want)


def held_small(got, oracle, D, F, h_eps):
    """test_gpu_moe.held for an fp32 output, with nothing absolute but what fp32 itself cannot hold: steps of 2^-149, of which
    F products and their parts each leave one."""
    want, inner, outer = oracle
    step = lambda n: (n / 32 + 24) * 2.0 ** -23  # noqa: E731
    bound = step(D) * inner + (step(F) + h_eps + 2.0 ** -18) * outer + 2.0 ** -24 * np.abs(want) + 4 * F * 2.0 ** -149
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= bound), f"{(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("form,w_codes", [("few", False), ("few", True), ("many", False)])   # (many, codes: not below 2^-57)
@pytest.mark.parametrize("factor", [1e-9, 1e-12, 1e-15, 1e-16])
def test_small_values_as_good_as_others(form, w_codes, factor):
    """x of these sizes gives h and outputs of their squares, down to 1e-33."""
    E, k, D, F, T = 2, 1, 64, 32, 12
    w, up, down = layer(E, 0, D, F, w_codes, 40)
    x, _, _ = rows(T, D, False, 41)
    ids, weights = pick(T, E, k, 42)
    x = (x.float() * factor).bfloat16()
    oracle = OS.moe(x.double().cpu().numpy(), ids, weights.astype(np.float64), up, down)
    got = S.moe_experts(x, torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), w, out_dtype=torch.float32, form=form)
    held_small(got, oracle, D, F, 2.0 ** -16 if form == "many" else 2.0 ** -22)
    # below what fp32 holds of h, 0 or the smallest values, and nothing that is not finite
    tiny = S.moe_experts((x.float() * 1e-16).bfloat16(), torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), w, out_dtype=torch.float32, form=form)
    assert tiny.abs().max() <= 1e-36


@pytest.mark.parametrize("w_codes", [False, True])
def test_small_and_large_values_in_one_row(w_codes):
    """A value of x or h 2^-30 of its row's largest, alone in a product, counts whole in the form for few tokens (with codes h
    in two parts keeps 2^-39 of the largest: 2^-9 of such a value, bf16 x all its bits)."""
    D, F = 64, 32
    up, down = torch.zeros((1, 2 * F, D)), torch.zeros((1, D, F))
    up[0, :F, 0], up[0, F:, 1] = 1, 1                # h_f = silu(x_0) x_1 ..
    up[0, 1, 0], up[0, 1, 2] = 0, 1                  # .. but for h_1 = silu(x_2) x_1
    down[0, 0, 0], down[0, 1, 1] = 1, 1
    x = torch.zeros((3, D))
    x[:, 0], x[:, 1], x[:, 2] = torch.tensor([30.0, 3.0, 100.0]), 1, 1.3125 * 2.0 ** -25
    if w_codes:
        code = lambda m: m.to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
        w = S.ExpertWeights(code(up), code(down), torch.ones((1, 2 * F), device="cuda"), torch.ones((1, D), device="cuda"))
    else:
        w = S.ExpertWeights(up.bfloat16().cuda(), down.bfloat16().cuda())
    got = S.moe_experts(x.bfloat16().cuda(), torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones((3, 1), device="cuda"), w,
                        out_dtype=torch.float32, form="few").double().cpu()
    xv = x.bfloat16().double()
    silu = lambda v: v / (1 + torch.exp(-v))  # noqa: E731
    eps = 2.0 ** -22 + 4 * 2.0 ** -24
    for i, g in ((0, xv[:, 0]), (1, xv[:, 2])):
        want = silu(g) * xv[:, 1]
        most = silu(xv[:, 0]) * xv[:, 1]
        assert torch.all((got[:, i] - want).abs() <= eps * want + (2.0 ** -22 * want + 2.0 ** -39 * most if w_codes else 0))
