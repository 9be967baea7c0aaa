"""csa2_sample where a block's piece of a row does not stay in shared memory and blocks are of 512 threads: some 20 rows and
more of vocabularies beyond 147,000 (fp32) and 294,000 (16 bits)."""
import pytest
import torch

from test_gpu_sample import check, draw

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


CUTS = [(0.9, 0, 1.0, 0.0), (1.1, 50, 0.9, 0.01), (1.0, 100000, 0.999, 0.0), (0.7, 0, 0.95, 0.0), (1.3, 700, 1.0, 0.0), (1.0, 0, 1.0, 0.02),
        (0.0, 0, 1.0, 0.0), (0.8, 512, 0.7, 0.0)]


@pytest.mark.parametrize("dtype,n,vocab", [("f32", 20, 150001), ("bf16", 20, 300001), ("f16", 20, 300007), ("f32", 32, 262144)])
def test_pieces_that_are_read_again(dtype, n, vocab):
    l, u = draw(n, vocab, dtype, 71)
    t, k, p, m = (list(v) for v in zip(*(CUTS[i % len(CUTS)] for i in range(n))))
    check(l, u, t, k, p, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_in_pieces_that_are_read_again(dtype):
    n, vocab = 20, 300032
    l, u = draw(n, vocab, dtype, 72)
    l[::2] = (l[::2].float() * 2).round().to(l.dtype) / 2       # steps of a half: thousands of equal logits
    check(l, u, None, [40000, 0, 3000, 7] * 5, [1.0, 0.6, 0.9, 0.5, 0.3] * 4, None)
