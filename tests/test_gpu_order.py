"""Calls in a row on one stream, without a wait between them: kernels that start before the one before them has ended read
nothing that is still being written."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Layer:
    """Query projection, router and sparse attention over tensors of their own; the query's place is the same in every call."""

    def __init__(self, T, window_only):
        N, K = 3000, 512
        inp = synth.make_inputs(synth.scaled(synth.WORKLOADS["batched_decode"], B=T, N=N), seed=41)
        rng = np.random.default_rng(42)
        dv = synth.to_device(inp)
        c, lay, rw, p = dv["cache"], dv["layers"][0], dv["rows"], dv["params"]
        idx = np.stack([np.sort(rng.choice(N, K, replace=False)) for _ in range(T)]).astype(np.int32)
        idx = torch.from_numpy(idx if not window_only else np.full((T, 0), 0, np.int32)).cuda()
        g = torch.Generator("cuda").manual_seed(43)
        rand = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
        self.xs = [rand(T, 4096, std=1.0) for _ in range(4)]
        self.x = self.xs[0].clone()
        self.proj = S.QueryProj(self.x, rand(1024, 4096, std=1 / 64), rand(64 * 512, 1024, std=1 / 32))
        self.route = S.ExpertRouter(self.x, rand(384, 4096, std=1 / 64), 6)
        self.args = (self.proj.q, rw["q_pos"], rw["seq_of_row"], c["lat"], c["lat_scales"], idx, lay["swa"], lay["swa_scale"],
                     rw["swa_pos0"], p["W"], lay["sink"], p["theta"], p["softmax_scale"])

    def attention(self):
        return S.sparse_attn(*self.args)[0]


def in_a_row(layer, between, attention):
    """The calls after a synchronisation each, and many times behind one another."""
    want = []
    for x in layer.xs:
        layer.x.copy_(x)
        layer.proj()
        torch.cuda.synchronize()
        for call in between:
            call()
        torch.cuda.synchronize()
        want.append(attention())
        torch.cuda.synchronize()
    for i in range(100):
        layer.x.copy_(layer.xs[i % 4])
        layer.proj()
        for call in between:
            call()
        got = attention()
        assert torch.equal(got, want[i % 4]), i


@pytest.mark.parametrize("T,window_only", [(1, False), (1, True), (32, False), (32, True)])
def test_attention_behind_the_projection_and_the_router(T, window_only):
    layer = Layer(T, window_only)
    in_a_row(layer, (layer.route,), layer.attention)


@pytest.mark.parametrize("T,window_only", [(1, False), (1, True), (32, False), (32, True), (320, False), (320, True)])
def test_attention_directly_behind_the_projection(T, window_only):
    layer = Layer(T, window_only)
    in_a_row(layer, (), layer.attention)


@pytest.mark.parametrize("T", [1, 32])
def test_partial_and_fused_attention_behind_the_projection(T):
    layer = Layer(T, False)
    in_a_row(layer, (), lambda: S.sparse_attn_partial(*layer.args[:10], *layer.args[11:])[0])
    q, q_pos, seq_of_row, lat, lat_scale, idx, swa, swa_scale, pos0, window, sink, theta, scale = layer.args
    reuse = S.DecodeLayer("reuse", seq_of_row=seq_of_row, n_visible=None, q=q, q_pos=q_pos, latents=lat, lat_scale=lat_scale, swa=swa,
                          swa_scale=swa_scale, swa_pos0=pos0, window=window, sink=sink, K=idx.shape[1], theta=theta, softmax_scale=scale, idx=idx)
    in_a_row(layer, (), lambda: reuse().clone())


@pytest.mark.parametrize("T", [1, 32])
def test_attentions_behind_one_another_over_one_workspace(T):
    """The second call's tiles over the window need nothing of the first's, whose partials are still being added up where
    theirs go (the caching allocator gives both the same workspace)."""
    layer = Layer(T, False)
    qs = []
    for x in layer.xs:
        layer.x.copy_(x)
        qs.append(layer.proj().clone())
    one = lambda q: S.sparse_attn(q, *layer.args[1:])[0]  # noqa: E731
    want = []
    for q in qs:
        torch.cuda.synchronize()
        want.append(one(q))
    torch.cuda.synchronize()
    for _ in range(25):
        got = [one(q) for q in qs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
