"""The workspaces of prepared router and experts calls among graph captures."""
import pytest
import torch

from test_gpu_moe import layer, pick, rows

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def inputs(T=3, E=4, k=2, D=128, F=64):
    w, _, _ = layer(E, 0, D, F, False, 50)
    x, _, _ = rows(T, D, False, 51)
    ids, weights = (torch.from_numpy(v).cuda() for v in pick(T, E, k, 52))
    return x, ids, weights, w


def test_one_made_within_a_capture_is_refused_in_another():
    x, ids, weights, w = inputs()
    router = torch.randn(4, 128, device="cuda").bfloat16()
    want, route = S.moe_experts(x, ids, weights, w), S.route_experts(x, router, 2)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        calls = S.MoEExperts(x, ids, weights, w), S.ExpertRouter(x, router, 2)
        for c in calls:
            c()
    still = torch.zeros(4, device="cuda")
    with torch.cuda.graph(second):  # (not run)
        still.add_(1)
        for c in calls:
            with pytest.raises(RuntimeError, match="capture"):
                c()
    for c in calls:
        with pytest.raises(RuntimeError, match="capture"):
            c()
    for _ in range(3):
        first.replay()
        assert torch.equal(calls[0].out, want) and torch.equal(calls[1].ids, route.ids) and torch.equal(calls[1].weights, route.weights)


def test_one_made_before_a_capture_without_a_synchronisation():
    """Counters whose zeros come late, on a stream that neither the capture nor the graph's runs wait for."""
    x, ids, weights, w = inputs()
    want = S.moe_experts(x, ids, weights, w)
    junk = torch.full((1 << 22,), 77, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        del junk
        one, two, three = (torch.cuda.Stream() for _ in range(3))
        with torch.cuda.stream(one):
            torch.cuda._sleep(20_000_000)
            call = S.MoEExperts(x, ids, weights, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(two):
            graph.capture_begin()
            call()
            call()
            graph.capture_end()
        with torch.cuda.stream(three):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out, want)
        del call, graph
        junk = torch.full((1 << 22,), 77, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()


def test_calls_while_another_thread_captures():
    """What a call asks about its zeros leaves a capture of another thread valid."""
    import threading
    x, ids, weights, w = inputs()
    want = S.moe_experts(x, ids, weights, w)
    call = S.MoEExperts(x, ids, weights, w)
    graph, begun, go_on, failed = torch.cuda.CUDAGraph(), threading.Event(), threading.Event(), []
    y = torch.zeros(8, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def capture():
        try:
            with torch.cuda.stream(one):
                graph.capture_begin()
                y.add_(1)
                begun.set()
                go_on.wait(60)
                y.add_(1)
                graph.capture_end()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
            begun.set()

    thread = threading.Thread(target=capture)
    thread.start()
    assert begun.wait(60)
    with torch.cuda.stream(two):
        for _ in range(3):
            call()
    go_on.set()
    thread.join()
    torch.cuda.synchronize()
    assert not failed, failed
    graph.replay()
    assert torch.equal(call.out, want) and (y == 2).all()
