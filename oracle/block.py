"""The operators next to the routed layer, in float64 (see the package docstring).

* the residual's addition and the root-mean-square norm,
* the activation encodings of the normed rows, given the scales,
* the router's logits and the product of 8-bit integers.

Steps whose rounding the kernels fix (the FP32 epilogue of the integer
product) are restated in float32; everything else is float64.
"""

import numpy as np

from . import formats as F


def rmsnorm(x, residual, weight, eps):
    """(h, y) in float64: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    with np.errstate(all="ignore"):
        root = np.sqrt(np.sum(h * h, axis=1, keepdims=True) / h.shape[1] + float(eps))
        return h, h / root * np.asarray(weight, dtype=np.float64)


def block_max(y, block):
    """Largest magnitude of every `block` consecutive columns: [M, H/block]."""
    M, H = y.shape
    return np.abs(y).reshape(M, H // block, block).max(axis=2)


def expand(scale, block):
    return np.repeat(scale, block, axis=1)


def mx_exponent(amax):
    """floor(log2 amax) - 8 clamped to [-127, 127]; -127 where amax is 0."""
    amax = np.asarray(amax, dtype=np.float64)
    _, e = np.frexp(amax)                      # amax = f 2^e, f in [1/2, 1)
    return np.where(amax > 0, np.clip(e - 1 - 8, -127, 127), -127)


def router_logits(x, w):
    return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T


def int8_sums(x, w):
    """Exact sums of products, int64 [M, N] (float64 holds them: |sum| < 2^31)."""
    return np.rint(x.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)


def int8_product(x, x_scale, w, w_scale, bias=None):
    """float32 [M, N]: the sum rounded to float32, times x_scale, times w_scale, plus bias, each step in float32."""
    acc = int8_sums(x, w).astype(np.float32)
    out = (acc * np.asarray(x_scale, np.float32)[:, None]).astype(np.float32)
    out = (out * np.asarray(w_scale, np.float32)[None, :]).astype(np.float32)
    if bias is not None:
        out = (out + np.asarray(bias, np.float32)[None, :]).astype(np.float32)
    return out


def e4m3_between(codes, lo, hi):
    """Whether each E4M3 code's value lies between the roundings of lo and hi (lo <= hi)."""
    v = F.e4m3_decode(codes)
    return (v >= F.e4m3_decode(F.e4m3_encode(lo))) & (v <= F.e4m3_decode(F.e4m3_encode(hi)))
