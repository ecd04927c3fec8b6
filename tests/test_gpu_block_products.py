"""moe_matmul_int8 and moe_router_logits against the oracle.

The integer product is compared bit for bit: the sum is exact and the
epilogue's FP32 steps are fixed.  The router's logits: products of two BF16
numbers are exact in FP32; an instruction adds 16 of them to the sum, each
such step and the joins of at most 8 partial sums erring by at most one FP32
step (2^-23) of the largest partial sum, itself at most sum |x w|, and the 16
products are aligned to the largest of them with as much lost each:
(H / 16 + 8 + 16) * 2^-23 * sum |x w|.
"""

import numpy as np
import pytest
import torch

from mixture_experts_routed_03_b200 import api, layer
from oracle import block as B
from oracle import formats as F
from tests.gpu_support import bf16_to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _status():
    return torch.zeros((1,), dtype=torch.int32, device=DEV)


def _codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int32).to(torch.int8)


def _case(M, N, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (_codes((M, K), g), torch.rand((M,), generator=g) + 0.01, _codes((N, K), g),
            (torch.rand((N,), generator=g) + 0.01) * 1e-3, torch.randn((N,), generator=g))


def _padded(t, stride):
    """The rows of t, `stride` elements apart, with codes that must not be read between them."""
    buf = torch.full((t.shape[0], stride), 77, dtype=t.dtype)
    buf[:, :t.shape[1]] = t
    return buf.to(DEV)


def _check(got, case, bias):
    x, xs, w, ws, b = case
    want = B.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), b.numpy() if bias else None)
    if got.dtype == torch.float32:
        assert np.array_equal(got.cpu().numpy(), want)
    else:
        assert np.array_equal(bf16_to_np(got), F.bf16_decode(F.bf16_encode(want)))


SHAPES = [(1, 1, 1), (1, 32, 128), (1, 1001, 4096), (2, 33, 100), (7, 31, 16), (8, 257, 1040), (9, 64, 144),
          (31, 255, 2048), (33, 96, 384), (64, 1536, 2048), (127, 130, 512), (128, 128, 128), (129, 300, 257),
          (200, 1, 640), (300, 1001, 1040), (513, 768, 2048), (1, 4096, 7168), (3000, 520, 256), (2500, 2500, 144),
          (1300, 1600, 272), (5000, 700, 400), (9473, 257, 130), (2400, 2104, 16), (12000, 129, 1040), (1281, 2305, 2048),
          (2, 1500, 2048), (2, 3000, 2050), (1, 500, 8192), (16, 4096, 7168), (64, 4096, 7168), (128, 4096, 7168),
          (256, 4096, 7168), (777, 7168, 2048), (2048, 4096, 512), (40, 64, 8192), (150, 200, 16384), (1000, 100, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_int8_product_bit_for_bit(M, N, K):
    case = _case(M, N, K, seed=M + N + K)
    stride = -(-K // 16) * 16 + 32
    x, w = _padded(case[0], stride), _padded(case[2], stride)
    xs, ws, b = case[1].to(DEV), case[3].to(DEV), case[4].to(DEV)
    status = _status()
    for fp32, bias in ((True, False), (False, True)):
        out = torch.empty((M, N), dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)
        api.matmul_int8(api.int8_problem(M, K, N, fp32, x_stride=stride, w_stride=stride), x, xs, w, ws, out, status,
                        bias=b if bias else None)
        _check(out, case, bias)
    assert int(status.item()) == api.MOE_OK


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,stride", [(5, 40, 48), (140, 129, 131), (140, 128, 132), (2, 30, 32), (4139, 1454, 1456),
                                        (2600, 2052, 2064), (3001, 2050, 2056)])
def test_int8_output_rows_apart_and_nothing_else_written(out_dtype, M, N, stride):
    case = _case(M, N, 256, seed=stride)
    buf = torch.full((M + 2, stride), 5.0, dtype=out_dtype, device=DEV)
    lin = layer.Int8Linear(case[2].to(DEV), case[3].to(DEV), case[4].to(DEV))
    out = buf[:M, :N]
    assert lin.forward(case[0].to(DEV), case[1].to(DEV), out=out) is out
    _check(out, case, True)
    assert (buf[M:] == 5).all() and (buf[:M, N:] == 5).all()
    lin.check_status()


def test_int8_largest_sums_do_not_overflow():
    K = 131071
    for sign in (-128, 127):
        x = torch.full((3, K), -128, dtype=torch.int8)
        w = torch.full((5, K), sign, dtype=torch.int8)
        case = (x, torch.ones(3), w, torch.ones(5), None)
        lin = layer.Int8Linear(w.to(DEV), torch.ones(5, device=DEV))
        xp = _padded(x, 131072)[:, :K]
        _check(lin.forward(xp, torch.ones(3, device=DEV), out_dtype=torch.float32), case, False)


def test_int8_long_reduction_sums_past_24_bits():
    """Sums whose low bits FP32 does not hold: exact up to the one rounding."""
    case = _case(4, 48, 8192, seed=2)
    x, w = case[0].abs().clamp(max=127), case[2].abs().clamp(max=127)
    case = (x, case[1], w, case[3], case[4])
    assert B.int8_sums(x.numpy(), w.numpy()).min() > 2 ** 24
    lin = layer.Int8Linear(w.to(DEV), case[3].to(DEV), case[4].to(DEV))
    _check(lin.forward(x.to(DEV), case[1].to(DEV), out_dtype=torch.float32), case, True)


def test_int8_single_row_of_odd_length():
    case = _case(1, 20, 77, seed=3)
    lin = layer.Int8Linear(case[2].to(DEV), case[3].to(DEV), case[4].to(DEV))
    _check(lin.forward(case[0].to(DEV), case[1].to(DEV)), case, True)


@pytest.mark.parametrize("M,N,K", [(3, 1, 1), (16, 100, 2048), (9, 1001, 100), (5, 17, 4096), (48, 255, 4096),
                                   (5, 1000, 4111), (24, 1, 131071), (9, 128, 16384), (24, 1000, 512), (300, 61, 15),
                                   (17, 1001, 2049), (300, 60, 7168), (64, 257, 4100), (24, 256, 16384), (13, 1000, 7175),
                                   (48, 60, 8192), (24, 100, 16399), (3, 2048, 2048), (31, 2048, 2048)])
@pytest.mark.parametrize("codes", ["any", "least", "ends"])
def test_int8_product_of_a_batch(M, N, K, codes):
    """The warps' MMAs at every split of K and height of tile; codes whose products and sums are the largest there are."""
    x, xs, w, ws, b = _case(M, N, K, seed=M + N)
    if codes == "least":
        x, w = torch.full_like(x, -128), torch.full_like(w, -128)
    elif codes == "ends":
        x, w = (torch.where(t < 0, -128, 127).to(torch.int8) for t in (x, w))
    stride = -(-K // 16) * 16
    out = torch.full((M + 1, N + 3), 5.0, device=DEV)
    status = _status()
    api.matmul_int8(api.int8_problem(M, K, N, True, x_stride=stride, w_stride=stride, out_stride=N + 3),
                    _padded(x, stride), xs.to(DEV), _padded(w, stride), ws.to(DEV), out, status, bias=b.to(DEV))
    _check(out[:M, :N], (x, xs, w, ws, b), True)
    assert (out[M] == 5).all() and (out[:M, N:] == 5).all() and int(status.item()) == api.MOE_OK


def test_int8_rows_that_end_with_their_memory():
    """Rows of odd length in memory that ends with the last of them: nothing behind it may matter."""
    M, N, K, stride = 9, 40, 141, 144
    x, xs, w, ws, b = _case(M, N, K, seed=41)
    bx, bw = (torch.full(((t.shape[0] - 1) * stride + K,), 99, dtype=torch.int8, device=DEV) for t in (x, w))
    for t, buf in ((x, bx), (w, bw)):
        torch.as_strided(buf, (t.shape[0], K), (stride, 1)).copy_(t)
    out = torch.empty((M, N), device=DEV)
    api.matmul_int8(api.int8_problem(M, K, N, True, x_stride=stride, w_stride=stride), bx, xs.to(DEV), bw, ws.to(DEV), out,
                    _status(), bias=b.to(DEV))
    _check(out, (x, xs, w, ws, b), True)


def test_int8_scales_that_are_not_finite_follow_the_arithmetic():
    case = _case(6, 40, 64, seed=4)
    xs = case[1].clone()
    xs[2], xs[3], xs[4] = float("nan"), 0.0, float("inf")
    lin = layer.Int8Linear(case[2].to(DEV), case[3].to(DEV), case[4].to(DEV))
    out = lin.forward(case[0].to(DEV), xs.to(DEV), out_dtype=torch.float32).cpu()
    assert torch.isnan(out[2]).all() and torch.equal(out[3], case[4])
    assert not torch.isfinite(out[4]).any()
    _check(out[[0, 1, 5]], (case[0][[0, 1, 5]], xs[[0, 1, 5]], case[2], case[3], case[4]), True)


def test_int8_two_streams_graphs_and_one_object():
    """Two captured calls of one object replayed side by side: they share the
    weights and the status word, and nothing else."""
    case = _case(96, 700, 1024, seed=5)
    lin = layer.Int8Linear(case[2].to(DEV), case[3].to(DEV), case[4].to(DEV))
    cases, graphs, outs, xs = [], [], [], []
    for s in range(2):
        c = _case(96, 700, 1024, seed=6 + s)
        c = (c[0], c[1], case[2], case[3], case[4])
        x, sc = torch.zeros_like(c[0]).to(DEV), c[1].to(DEV)
        lin.forward(x, sc)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = lin.forward(x, sc)
        x.copy_(c[0])
        cases.append(c), graphs.append(g), outs.append(out), xs.append((x, sc))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, c in zip(outs, cases):
        _check(out, c, True)
    lin.check_status()


# ------------------------------------------------------------------ router

def _router(M, E, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, H), generator=g).to(torch.bfloat16)
    w = (torch.randn((E, H), generator=g) * H ** -0.5).to(torch.bfloat16)
    return x, w


def _check_logits(got, x, w):
    want = B.router_logits(x.double().numpy(), w.double().numpy())
    size = B.router_logits(x.double().abs().numpy(), w.double().abs().numpy())
    H = x.shape[1]
    assert (np.abs(got.double().cpu().numpy() - want) <= (H / 16 + 8 + 16) * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("M,E,H", [(1, 1, 256), (1, 256, 7168), (3, 8, 256), (17, 60, 2048), (64, 256, 7168),
                                   (127, 65, 512), (130, 128, 4096), (777, 60, 2048), (300, 1024, 256),
                                   (4100, 33, 512), (1500, 1001, 768), (9000, 128, 1024), (16384, 60, 512),
                                   (20001, 300, 768), (3000, 256, 2048), (12345, 64, 4096), (2, 700, 2048),
                                   (4, 256, 7168), (5, 60, 2048), (8, 1000, 1024), (9, 256, 7168), (300, 256, 7168),
                                   (1000, 128, 4096), (4096, 256, 7168), (2000, 60, 2048), (3000, 20, 7168)])
def test_router_logits(M, E, H):
    x, w = _router(M, E, H, seed=M)
    buf = torch.full((M + 1, E), 3.0, device=DEV)
    status = _status()
    api.router_logits(api.problem(M, H, 128, E, 1), x.to(DEV), w.to(DEV), buf, status)
    _check_logits(buf[:M], x, w)
    assert (buf[M] == 3).all() and int(status.item()) == api.MOE_OK


@pytest.mark.parametrize("M,E,H", [(5, 1, 256), (48, 65, 512), (33, 1, 2816), (130, 60, 5120), (7, 1023, 5120),
                                   (16, 250, 2816), (24, 161, 4096), (5, 1, 8192), (9, 257, 7168), (777, 61, 256),
                                   (49, 1024, 1024), (31, 1023, 2816), (129, 250, 5120), (64, 256, 7168), (33, 513, 8192),
                                   (97, 160, 7168), (63, 64, 16384), (6, 7, 768), (65, 9, 1280), (9, 1023, 7168),
                                   (31, 250, 8192)])
def test_router_logits_of_a_batch(M, E, H):
    """The warps' MMAs at every split of K and height of tile, rows and experts that do not fill one."""
    x, w = _router(M, E, H, seed=M + E)
    buf = torch.full((M + 1, E), 3.0, device=DEV)
    status = _status()
    api.router_logits(api.problem(M, H, 128, E, 1), x.to(DEV), w.to(DEV), buf, status)
    _check_logits(buf[:M], x, w)
    assert (buf[M] == 3).all() and int(status.item()) == api.MOE_OK


@pytest.mark.parametrize("M,E,H", [(9, 40, 256), (64, 256, 7168), (40, 17, 4096)])
def test_router_values_that_are_not_finite_stay_in_their_row_and_column(M, E, H):
    """The last row and the last expert stand in for those past the ends: what they hold must not spread."""
    x, w = _router(M, E, H, seed=31)
    x[M - 1, H - 1], w[E - 1, 0], x[2, 5] = float("nan"), float("inf"), float("inf")
    out = torch.empty((M, E), device=DEV)
    api.router_logits(api.problem(M, H, 128, E, 1), x.to(DEV), w.to(DEV), out, _status())
    assert torch.isnan(out[M - 1]).all() and not torch.isfinite(out[2]).any() and not torch.isfinite(out[:, E - 1]).any()
    keep = [i for i in range(M - 1) if i != 2]
    _check_logits(out[keep][:, :E - 1], x[keep], w[:E - 1])


def test_router_batches_in_a_graph_beside_calls_on_another_stream():
    cases = [(_router(M, 256, 7168, seed=M), M) for M in (9, 64)]
    cases = [(x.to(DEV), w.to(DEV), torch.empty((M, 256), device=DEV), M) for (x, w), M in cases]
    status = _status()

    def run(case):
        x, w, out, M = case
        api.router_logits(api.problem(M, 7168, 128, 256, 1), x, w, out, status)

    for c in cases:
        run(c)
    want = [c[2].clone() for c in cases]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        for _ in range(5):
            run(cases[0])
    for c in cases:
        c[2].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            run(cases[1])
    torch.cuda.synchronize()
    assert torch.equal(cases[0][2], want[0]) and torch.equal(cases[1][2], want[1])


def test_products_of_many_shapes_one_after_the_other():
    """Calls of changing shapes back to back, two of each: nothing of one may reach the next."""
    import math
    import random
    rng = random.Random(5)

    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    status = _status()
    for _ in range(400):
        M, N, K = spread(1, 3000), spread(1, 1500), spread(1, 5000)
        if M * N * K > 2e9:
            continue
        if rng.random() < 0.5:
            E, H = min(N, 1024), 256 * max(1, K // 256)
            x = torch.randn((M, H), device=DEV).to(torch.bfloat16)
            w = torch.randn((E, H), device=DEV).to(torch.bfloat16)
            outs = [torch.full((M + 1, E), 7.0, device=DEV) for _ in range(2)]
            for o in outs:
                api.router_logits(api.problem(M, H, 128, E, 1), x, w, o, status)
            want, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
            assert ((outs[0][:M].double() - want).abs() <= (H / 16 + 24) * 2.0 ** -23 * size).all(), (M, E, H)
            assert torch.equal(outs[0], outs[1]) and (outs[0][M] == 7).all(), (M, E, H)
        else:
            stride, os = -(-K // 16) * 16 + 16 * rng.randrange(3), N + rng.randrange(9)
            x = torch.randint(-128, 128, (M, stride), device=DEV, dtype=torch.int32).to(torch.int8)
            w = torch.randint(-128, 128, (N, stride), device=DEV, dtype=torch.int32).to(torch.int8)
            xs, ws = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
            out = torch.full((M + 1, os), 7.0, device=DEV)
            for _ in range(2):
                api.matmul_int8(api.int8_problem(M, K, N, True, x_stride=stride, w_stride=stride, out_stride=os), x, xs,
                                w, ws, out, status)
            want = (x[:, :K].double() @ w[:, :K].double().t()).float() * xs[:, None] * ws[None, :]
            assert torch.equal(out[:M, :N], want), (M, N, K)
            assert (out[M] == 7).all() and (out[:M, N:] == 7).all(), (M, N, K, os)
    assert int(status.item()) == api.MOE_OK


def test_router_logits_same_bits_every_time():
    x, w = _router(64, 256, 7168, seed=9)
    x, w = x.to(DEV), w.to(DEV)
    status = _status()
    outs = [torch.empty((64, 256), device=DEV) for _ in range(4)]
    for o in outs:
        api.router_logits(api.problem(64, 7168, 128, 256, 1), x, w, o, status)
    assert all(torch.equal(outs[0], o) for o in outs)


def test_router_row_of_nan_stays_alone():
    x, w = _router(9, 16, 256, seed=10)
    x[4, 7] = float("nan")
    out = torch.empty((9, 16), device=DEV)
    api.router_logits(api.problem(9, 256, 128, 16, 1), x.to(DEV), w.to(DEV), out, _status())
    assert torch.isnan(out[4]).all()
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    _check_logits(out[keep], x[keep], w)


# ------------------------------------------------------------------ offsets past 32 bits, other work beside

def test_int8_output_past_32_bit_offsets():
    M, N, K = 270001, 8200, 16          # 2.2e9 outputs
    g = torch.Generator().manual_seed(11)
    rows = [0, 1, 262143, 262144, M - 2, M - 1]
    few, w = _codes((len(rows), K), g), _codes((N, K), g)
    ws = torch.rand((N,), generator=g)
    x = torch.zeros((M, K), dtype=torch.int8, device=DEV)
    xs = torch.ones((M,), device=DEV)
    x[rows] = few.to(DEV)
    out = layer.Int8Linear(w.to(DEV), ws.to(DEV)).forward(x, xs)
    _check(out[rows], (few, torch.ones(len(rows)), w, ws, None), False)
    assert not out[2:262143].any()


def test_router_rows_past_32_bit_offsets():
    M, E, H = 300003, 8, 8192           # 2.4e9 activations
    x, w = _router(4, E, H, seed=12)
    big = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    rows = [0, 262144, M - 2, M - 1]
    big[rows] = x.to(DEV)
    out = torch.empty((M, E), device=DEV)
    status = _status()
    api.router_logits(api.problem(M, H, 128, E, 1), big, w.to(DEV), out, status)
    _check_logits(out[rows], x, w)
    assert int(status.item()) == api.MOE_OK


@pytest.mark.parametrize("M", [1, 2, 8, 40, 700, 3000])
def test_products_beside_each_other_on_two_streams(M):
    """Both kinds at once, and of one kind two calls of different sizes: the
    streams share the SMs, their tensor memory and nothing else."""
    case = _case(M, 1200, 1024, seed=20 + M)
    lin = layer.Int8Linear(case[2].to(DEV), case[3].to(DEV), case[4].to(DEV))
    x, xs = case[0].to(DEV), case[1].to(DEV)
    rx, rw = _router(M, 96, 2048, seed=21 + M)
    gx, gw = rx.to(DEV), rw.to(DEV)
    logits, status = torch.empty((M, 96), device=DEV), _status()
    p = api.problem(M, 2048, 128, 96, 1)
    a, b = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        out = lin.forward(x, xs, stream=a)
        api.router_logits(p, gx, gw, logits, status, stream=b)
        small = lin.forward(x[:1], xs[:1], stream=b)
    torch.cuda.synchronize()
    _check(out, case, True)
    _check(small, (case[0][:1], case[1][:1]) + case[2:], True)
    _check_logits(logits, rx, rw)
    lin.check_status()
    assert int(status.item()) == api.MOE_OK


def test_overlapping_arguments_are_refused():
    buf = torch.zeros((64, 256), dtype=torch.int8, device=DEV)
    lin = layer.Int8Linear(torch.ones((16, 64), dtype=torch.int8, device=DEV), torch.ones(16, device=DEV))
    with pytest.raises(api.MoEError):
        lin.forward(buf[:, :64], torch.ones(64, device=DEV), out=buf.view(torch.bfloat16)[:, 64:80])
