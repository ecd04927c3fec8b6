"""The operators next to the layer run together, as a block uses them: norm,
router and routed layer in every format; norm with integer codes and the
integer product."""

import numpy as np
import pytest
import torch

from mixture_experts_routed_03_b200 import layer, workloads
from oracle import block as B
from oracle import moe as O
from tests.gpu_support import FLIP_FACTOR, TOL, bf16_half_ulp, bf16_to_np, device, rms, weights_of

pytestmark = pytest.mark.gpu


def _problem(fmt, M=24, shared=0):
    return workloads.problem("tiny_bf16", num_tokens=M, hidden=512, intermediate_hidden=256, num_experts=12,
                             num_topk=3, format=fmt, routing="logits", shared_expert=shared)


def _block(p, seed):
    dev = device()
    host = workloads.make_inputs(p, seed=seed, device="cpu")
    d = {k: (None if v is None else v.to(dev)) for k, v in host.items()}
    if p["format"] == "nvfp4":
        # rows quantised per token: the L1 scales are the weights' alone
        x_global = torch.tensor(workloads.X_STD / workloads.FP4_CODE_RMS)
        host["gate_up_expert_scales"] = host["gate_up_expert_scales"] / x_global
        d["gate_up_expert_scales"] = host["gate_up_expert_scales"].to(dev)
    g = torch.Generator().manual_seed(seed)
    M, H, E = p["num_tokens"], p["hidden"], p["num_experts"]
    x = (torch.randn((M, H), generator=g) * 0.5).to(torch.bfloat16).to(dev)
    r = torch.randn((M, H), generator=g).to(dev)
    w = (0.05 + 0.01 * torch.randn((H,), generator=g)).to(torch.bfloat16).to(dev)
    router = (torch.randn((E, H), generator=g) * 2).to(torch.bfloat16).to(dev)
    scale = torch.tensor([0.3 / 448], device=dev) if p["format"] == "fp8_tensor" else None
    return host, d, layer.MoELayer(p, weights_of(d), device=dev), x, r, w, router, scale


@pytest.mark.parametrize("fmt,shared", [("bf16", 0), ("fp8", 0), ("nvfp4", 0), ("mxfp8", 0), ("fp8_tensor", 0),
                                        ("fp8", 1)])
def test_norm_router_and_layer(fmt, shared):
    p = _problem(fmt, shared=shared)
    host, d, L, x, r, w, router, scale = _block(p, seed=4)
    out, res = L.forward_prenorm(x, w, router, residual=r, bias=d["bias"], x_scale=scale)
    torch.cuda.synchronize()
    L.check_status()
    # the steps one by one: the norm's codes and the logits have the same bits every time
    q, q_scale, rowwise, normed, res2 = L.norm_quantize(x, w, residual=r, x_scale=scale)
    assert torch.equal(res, res2)
    logits = L.router_logits(normed, router)
    idx, weights = L.route(logits, bias=d["bias"])
    inputs = {k: v for k, v in workloads.to_numpy(host).items() if not k.startswith("x")}
    inputs["x"] = q.view(torch.int16).cpu().numpy().view(np.uint16) if fmt == "bf16" else q.cpu().numpy()
    inputs["x_scale"] = None if q_scale is None else q_scale.cpu().numpy()
    inputs["x_row_scale"] = None if rowwise is None else rowwise.cpu().numpy().view(np.uint16)
    ref = O.moe_forward(p, inputs, idx.cpu().numpy(), weights.cpu().numpy())["out_f64"]
    got = bf16_to_np(out)
    assert rms(ref) > 0
    assert (np.abs(got - ref) <= FLIP_FACTOR * TOL[fmt] * rms(ref) + bf16_half_ulp(ref)).all()
    # and what the layer was given is the norm of the sum
    h, y = B.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), w.double().cpu().numpy(), np.float32(1e-6))
    assert np.abs(bf16_to_np(normed) - y).max() <= 2.0 ** -8 * np.abs(y).max() * (1 + 2.0 ** -10)
    want = B.router_logits(bf16_to_np(normed), router.double().cpu().numpy())
    size = B.router_logits(np.abs(bf16_to_np(normed)), router.double().abs().cpu().numpy())
    assert (np.abs(logits.double().cpu().numpy() - want) <= (512 / 16 + 24) * 2.0 ** -23 * size).all()


def test_block_in_a_graph_and_on_another_stream():
    p = _problem("mxfp8")
    host, d, L, x, r, w, router, _ = _block(p, seed=5)
    want, want_res = L.forward_prenorm(x, w, router, residual=r)
    side = torch.cuda.Stream(device())
    side.wait_stream(torch.cuda.current_stream())
    out, res = L.forward_prenorm(x, w, router, residual=r, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gout, gres = L.forward_prenorm(x, w, router, residual=r)
    graph.replay()
    torch.cuda.synchronize()
    L.check_status()
    a = bf16_to_np(want)
    for o, q in ((out, res), (gout, gres)):
        assert torch.equal(q, want_res)
        # the layer adds its FP32 rows in any order: 2^-20 of the sum of 3 terms, then one BF16 step
        assert (np.abs(bf16_to_np(o) - a) <= 2.0 ** -20 * np.abs(a).max() + 2 * bf16_half_ulp(a)).all()


def test_a_block_without_a_residual_hands_its_input_on():
    p = _problem("bf16", M=3)
    host, d, L, x, r, w, router, _ = _block(p, seed=6)
    out, res = L.forward_prenorm(x, w, router)
    assert res is x and out.shape == x.shape


def test_no_tokens():
    p = _problem("fp8", M=3)
    host, d, L, x, r, w, router, _ = _block(p, seed=7)
    out, res = L.forward_prenorm(x[:0], w, router, residual=r[:0])
    assert out.shape == (0, 512) and res.shape == (0, 512)


@pytest.mark.parametrize("M,H,N", [(1, 256, 40), (70, 1024, 513), (300, 2048, 256)])
def test_norm_codes_through_the_integer_product(M, H, N):
    dev = device()
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, H), generator=g).to(torch.bfloat16).to(dev)
    r = torch.randn((M, H), generator=g).to(torch.bfloat16).to(dev)
    w = torch.randn((H,), generator=g).to(torch.bfloat16).to(dev)
    wq = torch.randint(-127, 128, (N, H), generator=g, dtype=torch.int32).to(torch.int8).to(dev)
    ws = (torch.rand((N,), generator=g) + 0.1).to(dev) * 1e-3
    lin = layer.Int8Linear(wq, ws)
    n = layer.rmsnorm_quantize(x, w, r, "int8")
    out = lin.forward(n.codes, n.scales, out_dtype=torch.float32)
    lin.check_status()
    want = B.int8_product(n.codes.cpu().numpy(), n.scales.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
    assert np.array_equal(out.cpu().numpy(), want)
    # against the unquantised product: half a code step per element of the row, 2^-18 for the norm
    _, y = B.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), w.double().cpu().numpy(), np.float32(1e-6))
    real = y @ (wq.double().cpu().numpy() * ws.double().cpu().numpy()[:, None]).T
    step = n.scales.double().cpu().numpy()[:, None] * 0.5 * (1 + 2.0 ** -10)
    bound = step * np.abs(wq.double().cpu().numpy() * ws.double().cpu().numpy()[:, None]).sum(axis=1)[None, :]
    assert (np.abs(out.double().cpu().numpy() - real) <= bound * (1 + 2.0 ** -10) + 2.0 ** -16 * np.abs(y).sum(
        axis=1)[:, None] * 127 * ws.double().cpu().numpy()[None, :]).all()


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_a_block_beside_integer_products_on_another_stream(fmt):
    """The routed layer's kernels hold all tensor memory of an SM; the products
    on the other stream take what is free and neither waits for the other for good."""
    p = _problem(fmt, M=24)
    host, d, L, x, r, w, router, scale = _block(p, seed=8)
    want, want_res = L.forward_prenorm(x, w, router, residual=r, bias=d["bias"])
    dev = device()
    g = torch.Generator().manual_seed(9)
    wq = torch.randint(-127, 128, (700, 1024), generator=g, dtype=torch.int32).to(torch.int8)
    xq = torch.randint(-127, 128, (900, 1024), generator=g, dtype=torch.int32).to(torch.int8)
    lin = layer.Int8Linear(wq.to(dev), torch.ones(700, device=dev))
    gx, xs = xq.to(dev), torch.ones(900, device=dev)
    a, b = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for i in range(20):
        out, res = L.forward_prenorm(x, w, router, residual=r, bias=d["bias"], stream=a)
        prod = lin.forward(gx[:900 - 40 * i], xs[:900 - 40 * i], out_dtype=torch.float32, stream=b)
    torch.cuda.synchronize()
    L.check_status()
    lin.check_status()
    y = bf16_to_np(want)
    assert torch.equal(res, want_res)
    # FP32 rows added in any order: 2^-20 of the sum of 3 terms, then one BF16 step
    assert (np.abs(bf16_to_np(out) - y) <= 2.0 ** -20 * np.abs(y).max() + 2 * bf16_half_ulp(y)).all()
    assert np.array_equal(prod.cpu().numpy(), B.int8_sums(xq[:140].numpy(), wq.numpy()).astype(np.float32))
