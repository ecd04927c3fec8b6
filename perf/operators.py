"""The operators next to the routed layer, as one pass each: the residual's
addition with the root-mean-square norm and an 8-bit output, the router's
logits, and the matrix product in 8-bit integers.

With ``own`` false a pass is elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it is the call a user of the framework
makes.  ``exact`` restates each operator in 64 bits.
"""

import math

import torch

own = False

DEVICE = "cuda"
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one token of a decoding sequence through the norm before a small layer
        dict(name="norm_fp8_1", op="norm", tokens=1, hidden=2048, format="fp8", residual="bf16", norm_out=True),
        # a decode batch, microscaling codes for the experts, the normed row kept for the router
        dict(name="norm_mxfp8_64", op="norm", tokens=64, hidden=7168, format="mxfp8", residual="bf16",
             norm_out=True),
        # an odd number of prompt tokens, no residual yet (first block), one static scale
        dict(name="norm_fp8_tensor_1021", op="norm", tokens=1021, hidden=2048, format="fp8_tensor",
             residual="none", norm_out=False),
        # a whole prefill batch with the residual stream in 32 bits
        dict(name="norm_fp8_16384", op="norm", tokens=16384, hidden=4096, format="fp8", residual="fp32",
             norm_out=True),
        # router of a decode batch over many experts
        dict(name="router_64", op="router", tokens=64, hidden=7168, experts=256),
        # router of an odd-sized prompt, a number of experts that fills no tile
        dict(name="router_777", op="router", tokens=777, hidden=2048, experts=60),
        # router of a whole prefill batch
        dict(name="router_16384", op="router", tokens=16384, hidden=4096, experts=128),
        # one token through a dense gate and up projection: the weights are read once
        dict(name="int8_1", op="int8", tokens=1, k=7168, n=4096, out="bf16", bias=False),
        # a decode batch through a down projection
        dict(name="int8_64", op="int8", tokens=64, k=2048, n=7168, out="bf16", bias=False),
        # ragged in every size, 32-bit output
        dict(name="int8_333", op="int8", tokens=333, k=1040, n=1001, out="fp32", bias=True),
        # a whole prefill batch through a square projection
        dict(name="int8_16384", op="int8", tokens=16384, k=4096, n=4096, out="bf16", bias=True),
        # the two together: norm with codes for each token, then the product that reads them
        dict(name="norm_int8_product_2048", op="norm_product", tokens=2048, hidden=4096, n=1536, residual="bf16"),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "router", "int8", "int8", "norm_product"])
    tokens = _spread(rng, 1, 16384)
    if op == "norm":
        hidden = 256 * _spread(rng, 1, 32)
        tokens = min(tokens, 16384 * 4096 // hidden)
        return dict(op=op, tokens=tokens, hidden=hidden,
                    format=rng.choice(["bf16", "fp8", "mxfp8", "fp8_tensor"]),
                    residual=rng.choice(["none", "bf16", "fp32"]), norm_out=rng.random() < 0.5)
    if op == "router":
        return dict(op=op, tokens=tokens, hidden=256 * _spread(rng, 1, 28), experts=_spread(rng, 4, 512))
    if op == "int8":
        k = 16 * _spread(rng, 2, 512)
        n = _spread(rng, 16, 8192)
        tokens = max(1, min(tokens, 16384 * 4096 * 4096 // (k * n)))
        return dict(op=op, tokens=tokens, k=k, n=n, out=rng.choice(["bf16", "fp32"]), bias=rng.random() < 0.5)
    return dict(op=op, tokens=tokens, hidden=256 * _spread(rng, 1, 16), n=_spread(rng, 64, 4096),
                residual=rng.choice(["none", "bf16", "fp32"]))


def _stream_inputs(s, g, tokens, hidden, residual):
    """A block's output and the residual stream: a few channels far larger than the rest, as the stream has them."""
    loud = 1.0 + 15.0 * (torch.rand((hidden,), generator=g, device=DEVICE) < 0.01).float()
    s["x"] = (torch.randn((tokens, hidden), generator=g, device=DEVICE) * loud).to(torch.bfloat16)
    s["residual"] = None
    if residual != "none":
        r = torch.randn((tokens, hidden), generator=g, device=DEVICE) * (3.0 * loud)
        s["residual"] = r.to(torch.bfloat16) if residual == "bf16" else r
    s["norm_weight"] = (1.0 + 0.2 * torch.randn((hidden,), generator=g, device=DEVICE)).to(torch.bfloat16)


def _codes(shape, g):
    """8-bit integers as symmetric scales of a row's largest value leave them."""
    return (torch.randn(shape, generator=g, device=DEVICE) * 30.0).round_().clamp_(-127.0, 127.0).to(torch.int8)


def _weight_inputs(s, g, n, k, bias):
    s["w"] = _codes((n, k), g)
    s["w_scale"] = (0.5 + torch.rand((n,), generator=g, device=DEVICE)) * 1e-3
    s["bias"] = torch.randn((n,), generator=g, device=DEVICE) * 0.1 if bias else None


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = dict(case=dict(case))
    op, tokens = case["op"], case["tokens"]

    def buffer(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEVICE)

    if op == "norm":
        hidden, fmt = case["hidden"], case["format"]
        _stream_inputs(s, g, tokens, hidden, case["residual"])
        s["static_scale"] = None
        if fmt == "fp8_tensor":  # calibrated a little below the largest value that comes
            s["static_scale"] = torch.full((1,), 12.0 / E4M3_MAX, device=DEVICE)
        # the buffers of the calls' results, which a serving program keeps
        s["residual_out"] = None if s["residual"] is None else torch.empty_like(s["residual"])
        s["normed"] = buffer((tokens, hidden), torch.bfloat16) if case["norm_out"] or fmt == "bf16" else None
        s["codes"] = None if fmt == "bf16" else buffer((tokens, hidden), torch.uint8)
        s["scales"] = {"fp8": lambda: buffer((tokens, hidden // 128), torch.float32),
                       "mxfp8": lambda: buffer((tokens, hidden // 32), torch.uint8)}.get(fmt, lambda: None)()
    elif op == "router":
        hidden, experts = case["hidden"], case["experts"]
        s["x"] = torch.randn((tokens, hidden), generator=g, device=DEVICE).to(torch.bfloat16)
        s["router"] = (torch.randn((experts, hidden), generator=g, device=DEVICE) / math.sqrt(hidden)).to(
            torch.bfloat16)
        s["logits"] = buffer((tokens, experts), torch.float32)
    elif op == "int8":
        s["x"] = _codes((tokens, case["k"]), g)
        s["x_scale"] = (0.2 + torch.rand((tokens,), generator=g, device=DEVICE)) * 0.05
        _weight_inputs(s, g, case["n"], case["k"], case["bias"])
        s["out"] = buffer((tokens, case["n"]), torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    else:
        hidden = case["hidden"]
        _stream_inputs(s, g, tokens, hidden, case["residual"])
        _weight_inputs(s, g, case["n"], hidden, False)
        s["residual_out"] = None if s["residual"] is None else torch.empty_like(s["residual"])
        s["codes"] = buffer((tokens, hidden), torch.int8)
        s["scales"] = buffer((tokens,), torch.float32)
        s["out"] = buffer((tokens, case["n"]), torch.bfloat16)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEVICE)
    if own:  # the problem statements (sizes and formats, on the host), made once as the weights' owner does
        from mixture_experts_routed_03_b200 import api
        if op in ("norm", "norm_product"):
            s["norm_problem"] = api.norm_problem(tokens, hidden, case.get("format", "int8"), eps=EPS,
                                                 residual_fp32=case["residual"] == "fp32")
        if op in ("int8", "norm_product"):
            s["product_problem"] = api.int8_problem(tokens, case.get("k", case.get("hidden")), case["n"],
                                                    out_fp32=case.get("out") == "fp32")
        if op == "router":
            s["problem"] = api.problem(tokens, hidden, 128, experts, 1)
    return s


# ------------------------------------------------------------------ the plain form, in 32 bits

def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["norm_weight"].float()
    return (None if s["residual"] is None else h.to(s["residual"].dtype)), y


def _plain_codes(y, fmt, static_scale):
    """(codes, scales) of the normed rows: E4M3 codes as float8 values, scales as the numbers they are."""
    tokens, hidden = y.shape
    if fmt == "fp8_tensor":
        return (y * (1.0 / static_scale)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), None
    block = 128 if fmt == "fp8" else 32
    b = y.view(tokens, hidden // block, block)
    amax = b.abs().amax(dim=2)
    if fmt == "fp8":
        scale = amax / E4M3_MAX
        inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
        scales = scale
    else:  # frexp: amax = f 2^e with f in [1/2, 1), so floor(log2 amax) = e - 1
        exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
        inverse = torch.exp2(-exponent.float())
        scales = (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    q = (b * inverse[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(tokens, hidden), scales


def _plain_product(codes, x_scale, s, dtype):
    # sums of products of 8-bit integers: float32 holds their exact values or rounds them at 2^-24
    out = (codes.float() @ s["w"].float().t()) * x_scale[:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        out = out + s["bias"][None, :]
    return out.to(dtype)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        residual, y = _plain_norm(s)
        normed = y.to(torch.bfloat16) if s["normed"] is not None else None
        codes, scales = (None, None) if case["format"] == "bf16" else _plain_codes(y, case["format"],
                                                                                  s["static_scale"])
        return dict(residual=residual, normed=normed, codes=codes, scales=scales)
    if op == "router":
        return dict(logits=s["x"].float() @ s["router"].float().t())
    if op == "int8":
        return dict(out=_plain_product(s["x"], s["x_scale"], s, s["out"].dtype))
    residual, y = _plain_norm(s)
    scale = y.abs().amax(dim=1) / 127.0
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
    codes = (y * inverse[:, None]).round().clamp(-127.0, 127.0).to(torch.int8)
    return dict(residual=residual, scales=scale, out=_plain_product(codes, scale, s, torch.bfloat16))


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from mixture_experts_routed_03_b200 import api
    case = s["case"]
    op = case["op"]
    if op == "norm":
        api.rmsnorm_quantize(s["norm_problem"], s["x"], s["norm_weight"], residual_in=s["residual"],
                             residual_out=s["residual_out"], norm_out=s["normed"], codes=s["codes"],
                             scales=s["scales"], static_scale=s["static_scale"])
        codes, scales = s["codes"], s["scales"]
        if codes is not None:
            codes = codes.view(torch.float8_e4m3fn)
        if case["format"] == "mxfp8":
            scales = scales.view(torch.float8_e8m0fnu)
        return dict(residual=s["residual_out"], normed=s["normed"], codes=codes, scales=scales)
    if op == "router":
        api.router_logits(s["problem"], s["x"], s["router"], s["logits"], s["status"])
        return dict(logits=s["logits"])
    if op == "int8":
        api.matmul_int8(s["product_problem"], s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], s["status"],
                        bias=s["bias"])
        return dict(out=s["out"])
    api.rmsnorm_quantize(s["norm_problem"], s["x"], s["norm_weight"], residual_in=s["residual"],
                         residual_out=s["residual_out"], codes=s["codes"], scales=s["scales"])
    api.matmul_int8(s["product_problem"], s["codes"], s["scales"], s["w"], s["w_scale"], s["out"], s["status"])
    return dict(residual=s["residual_out"], scales=s["scales"], out=s["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ sizes of the work

def work(case):
    op, m = case["op"], case["tokens"]

    def norm(hidden, fmt, residual, normed):
        r = {"none": 0, "bf16": 2, "fp32": 4}[residual]
        codes = 0 if fmt == "bf16" else 1
        scales = {"fp8": 4 / 128, "mxfp8": 1 / 32}.get(fmt, 0)
        return m * hidden * (2 + 2 * r + codes + scales + (2 if normed or fmt == "bf16" else 0)) + 2 * hidden

    if op == "norm":
        return {"bytes": norm(case["hidden"], case["format"], case["residual"], case["norm_out"]),
                "flops": 8 * m * case["hidden"]}
    if op == "router":
        h, e = case["hidden"], case["experts"]
        return {"bytes": 2 * (m * h + e * h) + 4 * m * e, "flops": 2 * m * h * e}
    if op == "int8":
        k, n = case["k"], case["n"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + n * k + out * m * n + 4 * (m + n + (n if case["bias"] else 0)),
                "flops": 2 * m * k * n}
    h, n = case["hidden"], case["n"]
    return {"bytes": norm(h, "int8", case["residual"], False) - m * h + 4 * m + n * h + 4 * n + 2 * m * n,
            "flops": 8 * m * h + 2 * m * h * n}


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest_e4m3(v):
    """The E4M3 value nearest to each v: a step of 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6, at most 448."""
    exponent = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(s):
    total = s["x"].double()
    if s["residual"] is not None:
        total += s["residual"].double()
    root = torch.sqrt(torch.einsum("mh,mh->m", total, total) / total.shape[1] + EPS)
    return total, total / root[:, None] * s["norm_weight"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        return dict(logits=torch.einsum("mh,eh->me", s["x"].double(), s["router"].double()))
    if op == "int8":
        weight = s["w"].double() * s["w_scale"].double()[:, None]
        out = torch.einsum("mk,nk->mn", s["x"].double() * s["x_scale"].double()[:, None], weight)
        return dict(out=out if s["bias"] is None else out + s["bias"].double())
    total, y = _exact_norm(s)
    residual = None if s["residual"] is None else total
    if op == "norm_product":
        largest = y.abs().max(dim=1).values / 127.0
        codes = torch.round(y / largest[:, None])
        weight = s["w"].double() * s["w_scale"].double()[:, None]
        return dict(residual=residual, scales=largest, out=torch.einsum("mk,nk->mn", codes * largest[:, None], weight))
    normed = y if s["normed"] is not None else None
    fmt = case["format"]
    if fmt == "bf16":
        return dict(residual=residual, normed=normed, codes=None, scales=None)
    if fmt == "fp8_tensor":
        return dict(residual=residual, normed=normed, codes=_nearest_e4m3(y / s["static_scale"].double()), scales=None)
    blocks = y.unflatten(1, (-1, 128 if fmt == "fp8" else 32))
    largest = blocks.abs().max(dim=2).values
    scale = largest / E4M3_MAX if fmt == "fp8" else torch.exp2(torch.floor(torch.log2(largest)) - 8.0)
    return dict(residual=residual, normed=normed, codes=_nearest_e4m3(blocks / scale[:, :, None]).flatten(1),
                scales=scale)
