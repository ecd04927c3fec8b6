"""Failure detection of the products: an operand load or a finished sum that
never comes (withheld by a test hook) makes the bounded waits run out.  The
call returns within little more than one wait limit -- what is in flight is
waited for, but nothing waits a second limit -- with MOE_ERR_TIMEOUT in the
status word, and the next call is right.  Nothing faults or hangs the GPU."""

import time

import numpy as np
import pytest
import torch

from mixture_experts_routed_03_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LIMIT_US = 250000


def _call(kind, M, N, K):
    """(the call into a given output, what it should give)"""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    out = torch.empty((M, N), device=DEV)
    if kind == "router":
        x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
        w = torch.randn((N, K), generator=g, device=DEV).to(torch.bfloat16)
        p = api.problem(M, K, 128, N, 1)
        run = lambda: api.router_logits(p, x, w, out, status)  # noqa: E731
        want, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
        right = lambda: bool(((out.double() - want).abs() <= (K / 16 + 24) * 2.0 ** -23 * size).all())  # noqa: E731
    else:
        x = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
        w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
        xs, ws = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
        p = api.int8_problem(M, K, N, True)
        run = lambda: api.matmul_int8(p, x, xs, w, ws, out, status)  # noqa: E731
        want = (x.double() @ w.double().t()).float() * xs[:, None] * ws[None, :]
        right = lambda: torch.equal(out, want)  # noqa: E731
    return run, out, status, right


def _run_out(kind, M, N, K, hold):
    run, out, status, right = _call(kind, M, N, K)
    run()
    torch.cuda.synchronize()
    assert right() and int(status.item()) == api.MOE_OK
    out.fill_(7.0)
    torch.cuda.synchronize()
    try:
        api.product_test_hooks(LIMIT_US, hold)
        t0 = time.perf_counter()
        run()
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        api.product_test_hooks()
    left = out.clone()
    assert int(status.item()) == api.MOE_ERR_TIMEOUT
    assert LIMIT_US * 0.9e-6 < elapsed < LIMIT_US * 1.7e-6
    status.zero_()
    run()
    assert right() and int(status.item()) == api.MOE_OK
    return left


# one CTA a tile and K split over 2, 4 and 8; 64 to 256 columns; a ring that holds the whole share of K and one that does not
TILES = [("router", 8192, 256, 2048), ("router", 4736, 281, 6912), ("router", 1470, 125, 1280), ("router", 996, 132, 6144),
         ("int8", 333, 1001, 1040), ("int8", 352, 2147, 2576), ("int8", 274, 665, 5040), ("int8", 731, 63, 5728)]


@pytest.mark.parametrize("kind,M,N,K", TILES)
@pytest.mark.parametrize("hold", ["load", "sum"])
def test_tile_that_waits_in_vain_is_not_stored(kind, M, N, K, hold):
    left = _run_out(kind, M, N, K, hold)
    assert (left[0, :32] == 7).all()           # the first cluster's tile
    assert not (left[-1] == 7).all()           # others are


# CTA pairs: more tiles than pairs and fewer, every tile width; the second CTA's load is the one that its pair's first waits for
PAIRS = [(4096, 4096, 512), (2500, 2500, 144), (9473, 257, 130), (5000, 700, 400), (2048, 4096, 512), (16384, 4096, 1024)]


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("hold", ["load", "sum", "load_of_second"])
def test_pair_that_waits_in_vain(M, N, K, hold):
    K = -(-K // 16) * 16
    left = _run_out("int8", M, N, K, hold)
    assert (left == 7).any() and not (left == 7).all()      # the pair's last tile at least; the others' are stored


@pytest.mark.parametrize("kind,M,N,K", [("router", 4736, 281, 6912), ("int8", 274, 665, 5040)])
def test_second_cta_of_a_cluster_that_waits_in_vain(kind, M, N, K):
    assert (_run_out(kind, M, N, K, "load_of_second")[0, :32] == 7).all()


def test_hooks_are_part_of_a_captured_call_and_of_no_other():
    run, out, status, right = _call("router", 996, 132, 6144)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    try:
        api.product_test_hooks(20000, "load")
        with torch.cuda.graph(graph):
            run()
    finally:
        api.product_test_hooks()
    run()
    torch.cuda.synchronize()
    assert right() and int(status.item()) == api.MOE_OK
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == api.MOE_ERR_TIMEOUT
        status.zero_()
        run()
        torch.cuda.synchronize()
        assert right() and int(status.item()) == api.MOE_OK


def test_few_rows_have_no_waits_to_run_out():
    run, out, status, right = _call("int8", 1, 512, 512)
    try:
        api.product_test_hooks(1, "load")
        run()
    finally:
        api.product_test_hooks()
    assert right() and int(status.item()) == api.MOE_OK


def test_status_of_a_call_that_went_well_is_left_alone():
    run, out, status, right = _call("int8", 333, 1001, 1040)
    status.fill_(5)
    run()
    assert right() and np.array_equal(status.cpu().numpy(), [5])
