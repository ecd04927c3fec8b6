"""The router's logits keep their precision over long sums, in every kernel and
split, with products of both signs and of one, where truncation adds up: the
root mean square of the errors is below the bound of tests/router_precision.py."""

import pytest
import torch

from mixture_experts_routed_03_b200 import api
from tests import router_precision as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("shape", P.LONG, ids=lambda s: "-".join(map(str, s)))
def test_long_sums_keep_their_precision(shape, one_sign):
    M, E, H = shape[3:]
    g = torch.Generator(device=DEV).manual_seed(M + E + H)
    x = torch.randn((M, H), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((E, H), generator=g, device=DEV) * H ** -0.5).to(torch.bfloat16)
    if one_sign:
        x, w = x.abs(), w.abs()
    out = torch.empty((M, E), device=DEV)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    api.router_logits(api.problem(M, H, 128, E, 1), x, w, out, status)
    want = x.double() @ w.double().t()
    error = P.rms_error(out.double().cpu().numpy(), want.cpu().numpy())
    print(f"{shape} one sign {one_sign}: {error:.2e}")
    assert error < P.RMS and int(status.item()) == api.MOE_OK
