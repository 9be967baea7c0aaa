"""Rotary axes at far positions against angles of 60 decimal digits."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_csa2_gb300")

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("theta,R", [(10000.0, 64), (500000.0, 128), (1.0, 16), (3e7, 256)])
def test_far_positions(theta, R):
    getcontext().prec = 60
    pos = [0, 1, 2 ** 31, 2 ** 36 + 12345, 2 ** 40 - 1, -(2 ** 38) - 7, 2 ** 46 + 1, 2 ** 52 + 3]
    rng = np.random.default_rng(R)
    x = rng.standard_normal((len(pos), 2, R)).astype(np.float32)
    ref = np.empty(x.shape)
    for i in range(R // 2):
        turn = (Decimal(-2 * i) / R * Decimal(theta).ln()).exp() / TWO_PI
        for t, at in enumerate(pos):
            frac = at * turn % 1
            a = float(frac * TWO_PI)
            u, v = x[t, :, i].astype(np.float64), x[t, :, i + R // 2].astype(np.float64)
            ref[t, :, i], ref[t, :, i + R // 2] = u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a)
    got = S.rope_axes(torch.from_numpy(x).cuda(), torch.tensor(pos, device="cuda"), theta=theta).double().cpu().numpy()
    # the angle: |pos| * 2^-64 turns, 2^-33 of its fixed point, 2^-25 half turns in fp32 (2^-23.3 radians); sine,
    # cosine, two products and a sum 2^-23 each
    far = 2 * np.pi * (np.abs(np.array(pos, dtype=np.float64)) * 2.0 ** -64 + 2.0 ** -33)[:, None, None]
    size = np.abs(x).max(-1, keepdims=True)
    assert np.all(np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + 2 * size * (far + 2.0 ** -23.3 + 4 * 2.0 ** -23))


def test_tables_of_several_thetas_by_turns():
    x = torch.randn((3, 2, 64), device="cuda")
    pos = torch.tensor([5, 70, 1000], device="cuda")
    want = {}
    for _ in range(3):
        for theta in (1e4, 5e5, 1e6, 2e6, 3e6, 1e4):
            for R in (32, 64):
                got = S.rope_axes(x, pos, theta=theta, rot_dim=R)
                assert torch.equal(got, want.setdefault((theta, R), got))
    assert not torch.equal(want[1e4, 64], want[5e5, 64]) and not torch.equal(want[1e4, 32], want[1e4, 64])
