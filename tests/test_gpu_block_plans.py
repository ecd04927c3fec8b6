"""Every kernel, tile and split that the products' choice can take, once each
(tests/product_shapes.py): integers bit for bit, the router's logits against
float64, rows and columns behind the ends left as they were.

Logits: products of two BF16 numbers are exact in FP32, an MMA adds 16 of them
and a few-row kernel one at a time, each step at most 2^-23 of sum |x w| off,
and 24 more steps for the joins and the alignment within an MMA; the few-row
kernel's lanes take K / 32 steps of their own share each, at most K / 32 of the
whole."""

import pytest
import torch

from mixture_experts_routed_03_b200 import api
from tests.product_shapes import SHAPES, plan_key

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_every_choice(shape):
    kind, M, N, K = shape[0], *shape[5:]
    assert plan_key(kind, M, N, K) == shape[:5]          # on this device too
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if kind == "router":
        x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
        w = (torch.randn((N, K), generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
        out = torch.full((M + 1, N), 7.0, device=DEV)
        for _ in range(2):
            api.router_logits(api.problem(M, K, 128, N, 1), x, w, out, status)
        want, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
        steps = (K / 32 if shape[1] == "few" else K / 16) + 24
        assert ((out[:M].double() - want).abs() <= steps * 2.0 ** -23 * size).all()
        assert (out[M] == 7).all()
    else:
        stride = -(-K // 16) * 16 + 16
        x, w = (torch.randint(-128, 128, (n, stride), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
                for n in (M, N))
        xs, ws = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
        bias = torch.randn(N, generator=g, device=DEV)
        scaled = (x[:, :K].double() @ w[:, :K].double().t()).float() * xs[:, None] * ws[None, :]
        # rows of whole 16-byte pieces and rows of none, both types, with a bias and without
        for fp32, os, b in ((True, -(-N // 8) * 8, None), (True, N + 3, bias), (False, -(-N // 8) * 8, bias),
                            (False, N + 5, None)):
            out = torch.full((M + 1, os), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)
            api.matmul_int8(api.int8_problem(M, K, N, fp32, x_stride=stride, w_stride=stride, out_stride=os), x, xs, w,
                            ws, out, status, bias=b)
            want = scaled if b is None else scaled + b
            assert torch.equal(out[:M, :N], want.to(out.dtype))
            assert (out[M] == 7).all() and (out[:M, N:] == 7).all()
    assert int(status.item()) == api.MOE_OK
