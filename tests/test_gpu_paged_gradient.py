"""The rotation's gradient through autograd: against the formula's and differences, of strided and broadcast
tensors, of second order, captured; and the calls that would lose it."""
import numpy as np
import pytest
import torch

import oracle.paged as OP
from paged_testlib import TYPES, values

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _case(dtype, seed=0, T=9, H=3):
    rng = np.random.default_rng(seed)
    x, _ = values((T, H + 2, 64), rng, dtype)
    y, yd = values((T, H, 64), rng, dtype)
    pos = rng.integers(0, 5000, (2, T))
    return x.cuda(), y.cuda(), yd, pos, torch.from_numpy(pos).cuda(), rng


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pairing,inverse", [("half", False), ("adjacent", True)])
def test_gradient_against_the_formula(dtype, pairing, inverse):
    x, y, yd, pos, dpos, _ = _case(dtype)
    kw = dict(sections=(5, 11), theta=500.0, rot_dim=32, rot_first=16, pairing=pairing, inverse=inverse)
    x.requires_grad_(True)
    out = S.rope_axes(x[:, 1:4], dpos, **kw)
    with torch.no_grad():
        assert torch.equal(out, S.rope_axes(x[:, 1:4], dpos, **kw)) and not S.rope_axes(x[:, 1:4], dpos, **kw).requires_grad
    out.backward(y)
    ref = OP.rope_axes(yd, pos, [0] * 5 + [1] * 11, 500.0, 16, pairing == "half", not inverse)
    got = x.grad.double().cpu().numpy()
    # as the forward pass: sine, cosine, two products and a sum, 2^-23 each; the angle 2^-21.5
    size = np.abs(yd).max(-1, keepdims=True)
    assert np.all(np.abs(got[:, 1:4] - ref) <= EPS[dtype] * np.abs(ref) + 2 * size * (2.0 ** -21.5 + 4 * 2.0 ** -23))
    assert not got[:, [0, 4]].any()


def test_gradient_against_differences_and_of_second_order():
    x, y, _, _, pos, rng = _case("f32", 1, H=1)
    x = x[:, :1].contiguous().requires_grad_(True)
    f = lambda t: (S.rope_axes(t, pos, sections=(10, 22)) ** 2 * y).sum()  # noqa: E731
    g, = torch.autograd.grad(f(x), x, create_graph=True)
    v = torch.randn_like(x)
    gg, = torch.autograd.grad((g * v).sum(), x)
    with torch.no_grad():
        # sums of 9 * 64 squares times y: 2^-18 of their magnitude, twice, over the step
        size = float((S.rope_axes(x, pos, sections=(10, 22)) ** 2 * y.abs()).sum())
        for _ in range(10):
            i = tuple(int(rng.integers(n)) for n in x.shape)
            d = torch.zeros_like(x)
            d[i] = 0.25  # of second degree: central differences are exact but for rounding
            diff = (f(x + d).double() - f(x - d).double()).item() / 0.5
            assert abs(diff - g[i].item()) <= 2 * 2.0 ** -18 * size / 0.5
    # f is a quadratic form: its second derivative along v does not depend on x
    h, = torch.autograd.grad(f(v.requires_grad_(True)), v)
    assert float((gg - h).abs().max()) <= 2.0 ** -18 * float(h.abs().max())


def test_gradients_of_broadcast_and_misaligned_tensors():
    x, _, _, _, pos, _ = _case("f32", 2)
    x = x[:, :3].contiguous().requires_grad_(True)
    S.rope_axes(x, pos, sections=iter((16, 16))).sum().backward()
    want = S.rope_axes(torch.ones(x.shape, device="cuda"), pos, sections=(16, 16), inverse=True)
    assert torch.equal(x.grad, want)
    flat = torch.ones(x.numel() + 1, device="cuda")[1:].view(x.shape)  # 4 bytes behind an aligned address
    x.grad = None
    S.rope_axes(x, pos, sections=(16, 16)).backward(flat)
    assert torch.equal(x.grad, want)
    one = torch.randn((9, 1, 64), device="cuda", requires_grad=True)  # heads broadcast from one
    S.rope_axes(one.expand(9, 4, 64), pos, sections=(16, 16)).sum().backward()
    assert torch.allclose(one.grad, 4 * want[:, :1], rtol=0, atol=2.0 ** -20)


def test_calls_that_would_lose_the_gradient_are_refused():
    x, _, _, _, pos, _ = _case("bf16", 3)
    x = x[:, :3].contiguous().requires_grad_(True)
    with pytest.raises(ValueError):
        S.rope_axes(x, pos, sections=(16, 16), out=torch.empty_like(x))
    with pytest.raises(ValueError):
        S.rope_axes(x, pos, sections=(16, 16), out=x)
    with pytest.raises(ValueError):
        S.RopeAxes(x, pos, sections=(16, 16))
    with torch.no_grad():
        want = S.rope_axes(x, pos, sections=(16, 16))
        assert torch.equal(S.RopeAxes(x, pos, sections=(16, 16))(), want)
        assert torch.equal(S.rope_axes(x, pos, sections=(16, 16), out=torch.empty_like(x)), want)
    assert torch.equal(S.rope_axes(x.detach(), pos, sections=(16, 16)), want)


def test_captured_forward_and_backward():
    x, y, _, _, pos, _ = _case("f32", 4)
    x = x[:, :3].contiguous().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            S.rope_axes(x, pos, sections=(16, 16)).backward(y)
            x.grad = None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S.rope_axes(x, pos, sections=(16, 16))
        out.backward(y)
    for _ in range(3):
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
            y.copy_(torch.randn_like(y))
            x.grad.zero_()
        graph.replay()
        with torch.no_grad():
            assert torch.equal(out, S.rope_axes(x, pos, sections=(16, 16)))
            assert torch.equal(x.grad, S.rope_axes(y, pos, sections=(16, 16), inverse=True))
