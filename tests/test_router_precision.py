"""The bound on the router's logits (tests/router_precision.py) tells sums that
keep their precision from sums that do not: the arithmetic of the kernels
restated on the CPU, as it is and with mistakes in it."""

import numpy as np
import pytest

from mixture_experts_routed_03_b200 import api, build
from oracle import block as B
from tests import router_precision as P


def _inputs(H, one_sign, seed=0):
    rng = np.random.default_rng(seed)
    x, w = (np.float32(rng.standard_normal((n, H))) for n in (24, 32))
    x, w = ((a.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64) for a in (x, w))   # BF16
    return (np.abs(x), np.abs(w)) if one_sign else (x, w)


def _truncated(v):
    """v cut to 24 bits of mantissa, towards zero."""
    m, e = np.frexp(v)
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def _logits(x, w, mmas, partial=lambda v: v):
    """Sums of 16 products a step, cut after each; added to FP32 sums every `mmas` steps; `partial` of them joined."""
    total = np.zeros((x.shape[0], w.shape[0]))
    acc = np.zeros_like(total)
    for i in range(0, x.shape[1], 16):
        acc = _truncated(acc + _truncated(x[:, i:i + 16] @ w[:, i:i + 16].T))
        if (i // 16 + 1) % mmas == 0 or i + 16 == x.shape[1]:
            total = np.float32(total + np.float32(acc)).astype(np.float64)
            acc[:] = 0
    return partial(total)


@pytest.mark.parametrize("H", [2048, 16384])
@pytest.mark.parametrize("one_sign", [False, True])
def test_bound_holds_for_the_kernels_arithmetic(H, one_sign):
    x, w = _inputs(H, one_sign)
    assert P.rms_error(_logits(x, w, 16), B.router_logits(x, w)) < P.RMS


def test_bound_sees_a_sum_that_runs_on():
    x, w = _inputs(2048, True)
    assert P.rms_error(_logits(x, w, 128), B.router_logits(x, w)) > P.RMS


@pytest.mark.parametrize("one_sign", [False, True])
def test_bound_sees_partial_sums_of_16_bits(one_sign):
    x, w = _inputs(2048, one_sign)
    got = sum(_logits(x[:, i:i + 1024], w[:, i:i + 1024], 16, lambda v: v.astype(np.float16).astype(np.float64))
              for i in (0, 1024))
    assert P.rms_error(got, B.router_logits(x, w)) > 10 * P.RMS


@pytest.mark.parametrize("shape", P.LONG, ids=lambda s: "-".join(map(str, s)))
def test_long_shapes_take_their_kernels_and_are_long(shape):
    build.build()
    kernel, size, splits, M, E, H = shape
    p = api.product_plan(False, M, H, E)
    assert (api.PRODUCT_KERNELS[p.kernel], p.cols if kernel == "tiles" else p.rows, p.splits) == shape[:3]
    if kernel != "few":
        assert H // 16 // splits // (8 if kernel == "warps" else 1) >= 128
