"""csa2_add_norm with more rows than there are blocks: a block's next row is loaded while the present one is summed."""
import pytest
import torch

from test_gpu_norm import HALF, NORM, TYPES, rows, tiny

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def normed(s, gain, eps, offset=0.0):
    s = s.double()
    return s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * (gain.double() + offset)


# (rows, dim, stride, offset): about three rows to a block and no whole number of them; in 16-byte pieces with one, two and four
# to a thread, and value by value
SIZES = [(20011, 64, None, 0), (3001, 5120, None, 0), (5003, 2176, 2184, 8), (1003, 32768, None, 0), (15013, 77, None, 0),
         (1009, 2064, None, 1), (997, 8191, 8193, 3)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,dim,stride,offset", SIZES)
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_more_rows_than_blocks(dtype, n, dim, stride, offset, place):
    x = rows(n, dim, dtype, 61, stride, offset)
    gain = torch.linspace(-1, 2, dim, device="cuda")
    want = normed(x, gain, 1e-5)
    got = S.add_norm(x, gain, eps=1e-5, out=x if place == "in place" else None)
    assert (got.out.data_ptr() == x.data_ptr()) == (place == "in place")
    assert torch.all((got.out.double() - want).abs() <= (NORM + HALF[dtype]) * want.abs() + tiny(dtype))


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,dim,stride,offset", SIZES)
@pytest.mark.parametrize("place", ["apart", "in place", "into x"])
def test_sums_of_more_rows_than_blocks(dtype, stream, n, dim, stride, offset, place):
    if place == "into x" and dtype != stream:
        pytest.skip("another type than x")
    x, r = rows(n, dim, dtype, 62, stride, offset), rows(n, dim, stream, 63, stride, offset)
    total = (x.float() + r.float()).to(TYPES[stream])
    keep = x.clone(), r.clone()
    to = {"apart": torch.full((n, dim), 7.0, dtype=TYPES[stream], device="cuda"), "in place": None, "into x": x}[place]
    got = S.add_norm(x, None, residual=r, residual_out=to, out_dtype=torch.float32)
    assert torch.equal(got.residual_out, total)
    assert place == "into x" or torch.equal(x, keep[0])
    assert place == "in place" or torch.equal(r, keep[1])
    y = normed(total, torch.ones(dim, device="cuda"), 1e-6)
    assert torch.all((got.out.double() - y).abs() <= (NORM + HALF["f32"]) * y.abs())


@pytest.mark.parametrize("dtype,stream", [("bf16", None), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("n,dim,offset,group", [(20011, 64, 0, 32), (3001, 5120, 0, 0), (3001, 5120, 0, 128), (1003, 32768, 0, 256),
                                                (1009, 2064, 1, 16), (1009, 2064, 1, 0), (15013, 77, 0, 0)])
def test_codes_of_more_rows_than_blocks(dtype, stream, n, dim, offset, group):
    x = rows(n, dim, dtype, 64, offset=offset)
    x *= torch.linspace(0.01, 3, n, device="cuda").to(x.dtype)[:, None]    # rows that are told apart by their scales
    r = None if stream is None else rows(n, dim, stream, 65, offset=offset)
    s = x if r is None else (x.float() + r.float()).to(r.dtype)
    gain = torch.linspace(0.1, 3, dim, device="cuda")
    got = S.add_norm(x, gain, residual=r, quant_group=group, out_dtype=torch.float32)
    want = normed(s, gain, 1e-6)
    assert torch.all((got.out.double() - want).abs() <= (NORM + HALF["f32"]) * want.abs())
    # from the fp32 rows bit for bit: a division by 448 in 64 bits, rounded to fp32, is the fp32 quotient (53 bits are more
    # than twice 24 and two)
    y = got.out.reshape(n, -1, group or dim)
    scale = (y.abs().amax(-1).double() / 448).float()
    assert torch.equal(got.scales.reshape(scale.shape), scale)
    q = (y.double() / scale.double()[..., None]).float().to(torch.float8_e4m3fn)
    assert torch.equal(got.codes.reshape(y.shape), q.view(torch.uint8))


def test_a_sum_in_place_is_told_to_what_has_saved_it():
    x, r, w = torch.randn(3, 64, device="cuda"), torch.randn(3, 64, device="cuda"), torch.ones(64, device="cuda", requires_grad=True)
    y = (r * w).sum()
    S.add_norm(x, residual=r)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    call = S.AddNorm(x)
    y = (call().out * w).sum()
    y.backward()
    y = (call().out * w).sum()
    call()
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
