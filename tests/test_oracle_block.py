"""Pins of the float64 oracle of the operators next to the layer."""

import numpy as np
import torch

from oracle import block as B
from oracle import formats as F


def test_rmsnorm_against_torch_float64():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 512), generator=g, dtype=torch.float64)
    r = torch.randn((5, 512), generator=g, dtype=torch.float64)
    w = torch.randn((512,), generator=g, dtype=torch.float64)
    h, y = B.rmsnorm(x.numpy(), r.numpy(), w.numpy(), 1e-5)
    want = torch.nn.functional.rms_norm(x + r, (512,), w, 1e-5)
    assert np.array_equal(h, (x + r).numpy())
    assert np.allclose(y, want.numpy(), rtol=1e-13, atol=0)


def test_rmsnorm_of_a_constant_row_is_the_weight():
    w = np.linspace(-2, 2, 256)
    _, y = B.rmsnorm(np.full((1, 256), 3.0), None, w, 1e-300)
    assert np.allclose(y[0], w, rtol=1e-15, atol=0)


def test_mx_exponent_is_floor_log2():
    v = np.array([0.0, 1.0, 1.5, 2.0, np.nextafter(2.0, 0), 448.0, 2.0 ** -130, 3e38])
    assert B.mx_exponent(v).tolist() == [-127, -8, -8, -7, -8, 0, -127, 119]


def test_int8_sums_against_int64():
    rng = np.random.default_rng(0)
    x = rng.integers(-128, 128, (7, 333), dtype=np.int8)
    w = rng.integers(-128, 128, (5, 333), dtype=np.int8)
    assert np.array_equal(B.int8_sums(x, w), x.astype(np.int64) @ w.astype(np.int64).T)
    # the largest sum the product allows still fits 32 bits
    assert 131071 * 128 * 128 < 2 ** 31 <= 131072 * 128 * 128


def test_int8_product_rounds_like_torch_float32():
    rng = np.random.default_rng(1)
    x = rng.integers(-127, 128, (6, 64), dtype=np.int8)
    w = rng.integers(-127, 128, (4, 64), dtype=np.int8)
    xs, ws = rng.random(6).astype(np.float32), rng.random(4).astype(np.float32)
    b = rng.standard_normal(4).astype(np.float32)
    acc = torch.from_numpy(B.int8_sums(x, w)).float()
    want = acc * torch.from_numpy(xs)[:, None] * torch.from_numpy(ws)[None, :] + torch.from_numpy(b)[None, :]
    assert np.array_equal(B.int8_product(x, xs, w, ws, b), want.numpy())


def test_e4m3_between_accepts_the_rounding_and_nothing_else():
    v = np.array([0.3, 17.0, 447.0, 500.0, -0.001])
    c = F.e4m3_encode(v)
    assert B.e4m3_between(c, v, v).all()
    assert not B.e4m3_between(c ^ 1, v, v).any()
