"""moe_rmsnorm_quantize against the float64 oracle.

Tolerances, in units u = 2^-24 (half an FP32 step, relative).  h carries 1
rounding.  The FP32 sum of a warp's squares: 2 for h, 1 for the product or its
FMA, 3 for the sum of 8, at most 3 for a thread's 4 vectors, 5 for the lanes;
FP64 from there, so the mean is within 14 u, and the square root halves that:
rstd within 7 u.  y, for a scale or BF16: 7 + 1 for h, and at most 3 for
rstd's first part and two products: 11 u; a scale, the quotient of a maximum:
12 u.  A code's value: 8 u, its products' errors carried along (terms of order
u^2), 1 for the rounding of the result, and 2 between a block's scale and the
quotient that it is the rounding of.  All within 16 u = 2^-20, relative,
element by element.  What is rounded to
fewer bits must lie between the roundings of v (1 - 2^-20) and v (1 + 2^-20)
(rounding is monotonic); a code, of y / s with s the scale that the kernel
gave.
"""

import numpy as np
import pytest
import torch

from mixture_experts_routed_03_b200 import api, layer
from oracle import block as B
from oracle import formats as F
from tests.gpu_support import bf16_to_np

pytestmark = pytest.mark.gpu
Y_REL, CODE_REL = 2.0 ** -20, 2.0 ** -20
DEV = "cuda:0"
FORMATS = ["bf16", "fp8", "mxfp8", "fp8_tensor", "int8"]


def _inputs(M, H, residual="bf16", weight=torch.bfloat16, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    loud = 1 + 30 * (torch.rand((H,), generator=g) < 0.02).float()
    x = (torch.randn((M, H + pad), generator=g) * 0.7).to(torch.bfloat16)
    x[:, :H] *= loud.to(torch.bfloat16)
    r = None
    if residual:
        r = (torch.randn((M, H + pad), generator=g) * 2).to(torch.bfloat16 if residual == "bf16" else torch.float32)
    w = (1 + 0.3 * torch.randn((H,), generator=g)).to(weight)
    return (x.to(DEV)[:, :H], None if r is None else r.to(DEV)[:, :H], w.to(DEV),
            torch.tensor([0.03], device=DEV))


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _between_bf16(got, y, rel):
    lo, hi = np.minimum(y * (1 - rel), y * (1 + rel)), np.maximum(y * (1 - rel), y * (1 + rel))
    return (got >= F.bf16_decode(F.bf16_encode(lo))) & (got <= F.bf16_decode(F.bf16_encode(hi)))


def _ends(v, rel):
    return np.minimum(v * (1 - rel), v * (1 + rel)), np.maximum(v * (1 - rel), v * (1 + rel))


def check(out, x, residual, weight, static_scale, fmt, eps):
    h, y = B.rmsnorm(_f64(x), _f64(residual), _f64(weight), np.float32(eps))
    M, H = h.shape
    if residual is not None and out.residual is not None:
        if residual.dtype == torch.float32:
            assert np.array_equal(_f64(out.residual), h.astype(np.float32).astype(np.float64))
        else:
            assert _between_bf16(bf16_to_np(out.residual), h, 2.0 ** -24).all()
    if out.norm is not None:
        assert _between_bf16(bf16_to_np(out.norm), y, Y_REL).all()
    if fmt == "bf16":
        assert out.codes is None and out.scales is None
        return
    codes = out.codes.cpu().numpy()
    if fmt == "fp8_tensor":
        v = y / np.float64(static_scale.item())
    elif fmt == "fp8":
        s = _f64(out.scales)
        want = B.block_max(y, 128) / 448.0
        assert (np.abs(s - want) <= CODE_REL * want).all()
        v = y / B.expand(s, 128)
    elif fmt == "mxfp8":
        X = out.scales.cpu().numpy().astype(np.int64) - 127
        amax = B.block_max(y, 32)
        assert ((X >= B.mx_exponent(amax * (1 - Y_REL))) & (X <= B.mx_exponent(amax * (1 + Y_REL)))).all()
        v = y * B.expand(np.ldexp(1.0, -X), 32)
    else:
        s = _f64(out.scales)
        want = np.abs(y).max(axis=1) / 127.0
        assert s.shape == (M,) and (np.abs(s - want) <= CODE_REL * want).all()
        lo, hi = _ends(y / s[:, None], CODE_REL)
        assert ((codes >= np.rint(lo)) & (codes <= np.rint(hi)) & (codes >= -127)).all()
        return
    lo, hi = _ends(v, CODE_REL)
    assert B.e4m3_between(codes, lo, hi).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,H", [(1, 256), (3, 512), (7, 1280), (130, 1024), (5, 2048), (2, 4096), (3, 7168), (2, 8192),
                                 (2, 8448), (1, 16384), (2, 32768)])
def test_against_oracle(fmt, M, H):
    for residual, weight in ((None, torch.bfloat16), ("bf16", torch.float32), ("fp32", torch.bfloat16)):
        x, r, w, ss = _inputs(M, H, residual, weight, seed=M + H)
        out = layer.rmsnorm_quantize(x, w, r, fmt, 1e-5, ss if fmt == "fp8_tensor" else None, norm=True)
        check(out, x, r, w, ss, fmt, 1e-5)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tokens(fmt):
    x, r, w, ss = _inputs(2051, 768, "fp32", torch.float32, seed=3)
    out = layer.rmsnorm_quantize(x, w, r, fmt, 1e-6, ss if fmt == "fp8_tensor" else None, norm=fmt != "fp8")
    check(out, x, r, w, ss, fmt, 1e-6)


@pytest.mark.parametrize("residual", ["bf16", "fp32"])
def test_strided_rows_and_in_place_residual(residual):
    x, r, w, ss = _inputs(9, 1536, residual, seed=5, pad=64)
    assert x.stride(0) == 1600
    kept = r.clone()
    behind = torch.as_strided(r, (9, 64), (1600, 1), r.storage_offset() + 1536).clone()
    out = layer.rmsnorm_quantize(x, w, r, "fp8", residual_out=r)
    assert out.residual is r
    check(out, x, kept, w, ss, "fp8", 1e-6)
    # what lies between the rows is left as it was
    assert torch.equal(torch.as_strided(r, (9, 64), (1600, 1), r.storage_offset() + 1536), behind)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nothing_written_behind_the_last_token(fmt):
    M, H = 3, 512
    x, r, w, ss = _inputs(M, H, seed=6)
    res = torch.full((M + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    norm = torch.full((M + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((M + 2, H), 99, dtype=torch.uint8, device=DEV)
    scales = torch.full((M + 2, H // 32 * 4), 99, dtype=torch.uint8, device=DEV)
    plain = fmt == "bf16"
    api.rmsnorm_quantize(api.norm_problem(M, H, fmt), x, w, residual_in=r, residual_out=res, norm_out=norm,
                         codes=None if plain else codes, scales=None if plain or fmt == "fp8_tensor" else scales,
                         static_scale=ss if fmt == "fp8_tensor" else None)
    torch.cuda.synchronize()
    assert (res[M:] == 7).all() and (norm[M:] == 7).all() and (codes[M:] == 99).all()
    used = {"fp8": M * (H // 128) * 4, "mxfp8": M * (H // 32), "int8": M * 4}.get(fmt, 0)
    assert (scales.view(-1)[used:] == 99).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_zeros_tiny_and_large_values(fmt):
    H = 512
    x, _, w, ss = _inputs(6, H, None, seed=7)
    x = x.contiguous()
    x[0] = 0
    x[1] *= 2.0 ** -60          # far below eps: y is tiny
    x[2] = 0
    x[2, 5] = 3.0               # one value: every other block is zeros
    x[3] *= 2.0 ** 50
    x[4] = 2.0 ** -133          # subnormal BF16
    out = layer.rmsnorm_quantize(x, w, None, fmt, 1e-6, ss if fmt == "fp8_tensor" else None, norm=True)
    keep = [1, 2, 3, 5]
    sub = type(out)(*[None if t is None else t[keep] for t in out])
    if fmt in ("fp8", "mxfp8"):
        codes = out.codes.view(6, -1, 128 if fmt == "fp8" else 32)
        assert not (codes[2, 1:] & 0x7F).any() and not out.scales[2, 1:].any()
        # a block of zeros has scale 0 and codes 0: nothing to divide by in the comparison below
        first = type(out)(out.codes[2:3, :32 if fmt == "mxfp8" else 128], out.scales[2:3, :1], None, None)
        assert (first.codes & 0x7F).sum() > 0
        keep = [1, 3, 5]
        sub = type(out)(*[None if t is None else t[keep] for t in out])
    check(sub, x[keep], None, w, ss, fmt, 1e-6)
    assert not out.norm[0].any()
    if fmt != "bf16":
        assert not (out.codes[0].view(torch.uint8) & 0x7F).any()
    if fmt in ("fp8", "int8"):
        assert not out.scales[0].any()
    if fmt == "mxfp8":
        assert not out.scales[0].any()      # 2^-127


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_are_not_finite_become_nan_and_stay_alone(fmt, bad):
    """3e38 squared leaves FP32: its row counts as not finite too."""
    x, r, w, ss = _inputs(5, 768, "fp32", seed=8)
    x = x.contiguous()
    r[2, 100] = bad
    out = layer.rmsnorm_quantize(x, w, r, fmt, 1e-6, ss if fmt == "fp8_tensor" else None, norm=True)
    assert torch.isnan(out.norm[2]).all()
    if fmt == "int8":
        assert not out.codes[2].any() and torch.isnan(out.scales[2])
    elif fmt != "bf16":
        assert ((out.codes[2] & 0x7F) == 0x7F).all()
    if fmt == "fp8":
        assert torch.isnan(out.scales[2]).all()
    if fmt == "mxfp8":
        assert (out.scales[2] == 255).all()
    keep = [0, 1, 3, 4]
    check(type(out)(*[None if t is None else t[keep] for t in out]), x[keep], r[keep], w, ss, fmt, 1e-6)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "int8", "fp8_tensor"])
def test_a_weight_that_is_not_finite_stays_in_its_block(fmt):
    x, _, w, ss = _inputs(2, 512, None, seed=9)
    w = w.clone()
    w[130] = float("nan")
    out = layer.rmsnorm_quantize(x, w, None, fmt, 1e-6, ss if fmt == "fp8_tensor" else None)
    if fmt == "int8":
        assert torch.isnan(out.scales).all() and not out.codes.any()
        return
    nan = (out.codes & 0x7F) == 0x7F
    block = {"fp8": 128, "mxfp8": 32, "fp8_tensor": 1}[fmt]
    at = torch.arange(512, device=DEV) // block == 130 // block
    assert nan[:, at].all() and not nan[:, ~at].any()


@pytest.mark.parametrize("value", [0.0, -1.0, float("nan"), float("inf"), 1e-40])
def test_static_scale_that_is_no_scale_gives_nan_codes(value):
    x, _, w, _ = _inputs(2, 256, None, seed=10)
    out = layer.rmsnorm_quantize(x, w, None, "fp8_tensor", static_scale=torch.tensor([value], device=DEV))
    assert ((out.codes & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("value", [1e-6, 2.0 ** -126])
def test_saturates_at_the_largest_code(value):
    x, _, w, _ = _inputs(4, 256, None, seed=11)
    out = layer.rmsnorm_quantize(x, w, None, "fp8_tensor", static_scale=torch.tensor([value], device=DEV))
    assert ((out.codes & 0x7F) == 0x7E).all()


def test_codes_are_those_of_the_exact_values():
    """2^20 values: a code differs from the exact value's only at a midpoint,
    within 2^-21 of it.  Spread evenly over a code's width (2^-3 to 2^-4 of
    it, both of whose ends count), at most 2 * 16 * 2^-21 of them lie so near:
    16 expected at most, 48 allowed (8 standard deviations above 16)."""
    x, r, w, ss = _inputs(256, 4096, "fp32", torch.float32, seed=17)
    out = layer.rmsnorm_quantize(x, w, r, "fp8_tensor", static_scale=ss)
    _, y = B.rmsnorm(_f64(x), _f64(r), _f64(w), np.float32(1e-6))
    want = F.e4m3_encode(y / np.float64(ss.item()))
    assert (out.codes.cpu().numpy() != want).sum() <= 48


def test_mxfp8_exponent_clamp():
    """A row under a tiny weight: amax below 2^-119, whose exponent is clamped at -127."""
    x, _, w, ss = _inputs(2, 256, None, torch.float32, seed=12)
    w = w * 2.0 ** -122
    out = layer.rmsnorm_quantize(x, w, None, "mxfp8")
    check(out, x, None, w, ss, "mxfp8", 1e-6)
    assert (out.scales == 0).any()


def test_int8_scale_below_the_smallest_normal_is_zero():
    x, _, w, _ = _inputs(2, 256, None, torch.float32, seed=13)
    for fmt in ("int8", "fp8"):
        out = layer.rmsnorm_quantize(x, w * 2.0 ** -130, None, fmt)
        assert not out.scales.any() and not (out.codes.view(torch.uint8) & 0x7F).any()


def test_graph_replay_and_another_stream():
    x, r, w, ss = _inputs(33, 2048, "bf16", seed=14)
    x = x.contiguous()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    eager = layer.rmsnorm_quantize(x, w, r, "mxfp8", norm=True, stream=side)
    side.synchronize()
    check(eager, x, r, w, ss, "mxfp8", 1e-6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.rmsnorm_quantize(x, w, r, "mxfp8", norm=True)
    x.copy_(_inputs(33, 2048, "bf16", seed=15)[0])
    graph.replay()
    torch.cuda.synchronize()
    check(out, x, r, w, ss, "mxfp8", 1e-6)


def test_the_same_bits_every_time():
    x, r, w, _ = _inputs(64, 7168, "bf16", seed=16)
    a = layer.rmsnorm_quantize(x, w, r, "int8", norm=True)
    for _ in range(3):
        b = layer.rmsnorm_quantize(x, w, r, "int8", norm=True)
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
    # and a token's result does not depend on its neighbours
    one = layer.rmsnorm_quantize(x[5:6], w, r[5:6], "int8", norm=True)
    assert all(torch.equal(p[5:6].view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, one))


@pytest.mark.parametrize("fmt,H", [("int8", 16384), ("mxfp8", 16384), ("fp8", 512)])
def test_offsets_past_32_bits(fmt, H):
    M = (1 << 31) // H + 5
    x, _, w, ss = _inputs(4, H, None, seed=18)
    rows = [0, 7, M - 2, M - 1]
    big = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    big[rows] = x
    out = layer.rmsnorm_quantize(big, w, None, fmt)
    check(type(out)(*[None if t is None else t[rows] for t in out]), x, None, w, ss, fmt, 1e-6)
    assert not (out.codes[100:200].view(torch.uint8) & 0x7F).any()


@pytest.mark.parametrize("fmt,M,H,residual", [("fp8", 1801, 7168, "bf16"), ("mxfp8", 2100, 4096, "fp32"),
                                              ("int8", 3300, 8192, None), ("bf16", 401, 32768, "bf16"),
                                              ("fp8_tensor", 12400, 1024, "bf16")])
def test_many_long_rows_in_place(fmt, M, H, residual):
    """Inputs past 48 MB, of which blocks ask L2 for the rows to come, in place and to the last row of their memory."""
    rows = [0, 1, M // 2, M - 2, M - 1]
    part, r, w, ss = _inputs(len(rows), H, residual, seed=23)
    x = torch.randn((M, H), device=DEV).to(torch.bfloat16)
    x[rows] = part
    stream = None
    if residual:
        stream = torch.randn((M, H), device=DEV).to(r.dtype)
        stream[rows] = r
    out = layer.rmsnorm_quantize(x, w, stream, fmt, 1e-6, ss if fmt == "fp8_tensor" else None, residual_out=stream)
    check(type(out)(*[None if t is None else t[rows] for t in out]), part, r, w, ss, fmt, 1e-6)


def test_residual_of_the_other_rows_is_untouched_in_place():
    """In place on a slice of a longer stream: the tokens before and behind keep theirs."""
    x, r, w, ss = _inputs(40, 1024, "bf16", seed=19)
    kept = r.clone()
    part = r[8:30]
    out = layer.rmsnorm_quantize(x[8:30], w, part, "fp8", residual_out=part)
    assert torch.equal(r[:8], kept[:8]) and torch.equal(r[30:], kept[30:])
    check(out, x[8:30], kept[8:30], w, ss, "fp8", 1e-6)


def test_overlapping_arguments_are_refused():
    x, r, w, _ = _inputs(8, 512, "bf16", seed=20)
    with pytest.raises(api.MoEError):
        layer.rmsnorm_quantize(x, w, r, "fp8", residual_out=x)
    longer = torch.cat([r, r[:1]])
    with pytest.raises(api.MoEError):
        layer.rmsnorm_quantize(x, w, longer[:8], "fp8", residual_out=longer[1:])
