"""A routed-MoE layer object over the C ABI: owns the device workspace and the
prepared weight blobs (the tensor-core tile layout ``moe_prepare_weights``
writes once, NVFP4 scale tiles included), and forwards calls to ``api``.

torch supplies device memory and streams only; every step runs in the
library's kernels.

The operators next to the layer are here too: ``rmsnorm_quantize`` (residual
addition, RMS norm and activation encoding), ``Int8Linear`` (a dense product
in 8-bit integers) and, on the layer itself, ``router_logits`` and
``forward_prenorm``, which runs norm, router and layer in a row.
"""

import collections
import contextlib

import torch

from . import api


def _i32(n, device):
    return torch.empty(max(int(n), 1), dtype=torch.int32, device=device)


@contextlib.contextmanager
def _on(device, stream):
    """The device made current, and with it `stream` (a torch stream, a raw
    cudaStream_t or None for the device's current one), so that buffers
    allocated inside belong to the stream that uses them."""
    with torch.cuda.device(device):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            yield


def _expect(name, t, dtypes, shape, device=None):
    """t is a tensor of one of the dtypes and of this shape, its rows dense, on the device."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or tuple(t.shape) != tuple(shape):
        got = (t.dtype, tuple(t.shape)) if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} {tuple(shape)}, got {got}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows that overlap (an expanded tensor?) are not taken")
    if device is not None and (t.device.type != device.type or device.index not in (None, t.device.index)):
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _row_stride(t, multiple=1):
    """Elements from one row to the next; of a single row, whose stride says
    nothing, its length rounded up to `multiple`."""
    if t.shape[0] > 1:
        return t.stride(0)
    return -(-t.shape[1] // multiple) * multiple


NormOutput = collections.namedtuple("NormOutput", "codes scales norm residual")


def rmsnorm_quantize(x, weight, residual=None, format="bf16", eps=1e-6, static_scale=None, norm=False,
                     residual_out=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; y encoded
    (see moe_rmsnorm_quantize in include/moe.h).

    x:            BF16 [M, H], rows any multiple of 16 bytes apart
    weight:       BF16 or FP32 [H]
    residual:     BF16 or FP32 [M, H], or None
    format:       "bf16", "fp8", "mxfp8", "fp8_tensor" (with static_scale, FP32 [1]) or "int8"
    norm:         also return y in BF16 (always, for "bf16")
    residual_out: where h goes; None allocates it, `residual` updates it in place
    Returns NormOutput(codes uint8 or int8 [M, H], scales, norm BF16 [M, H], residual), None where there is none.
    """
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a tensor [M, H]")
    M, H = x.shape
    _expect("x", x, (torch.bfloat16,), (M, H))
    dev = x.device
    _expect("weight", weight, (torch.bfloat16, torch.float32), (H,), dev)
    if residual is not None:
        _expect("residual", residual, (torch.bfloat16, torch.float32), (M, H), dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if residual_out is not None:
        _expect("residual_out", residual_out, (residual.dtype,), (M, H), dev)
    if static_scale is not None:
        _expect("static_scale", static_scale, (torch.float32,), (1,), dev)
    if format not in api.NORM_FORMATS:
        raise ValueError(f"format {format!r}: expected one of {', '.join(api.NORM_FORMATS)}")
    with _on(dev, stream):
        if residual is not None and residual_out is None:
            residual_out = torch.empty((M, H), dtype=residual.dtype, device=dev)
        y = torch.empty((M, H), dtype=torch.bfloat16, device=dev) if norm or format == "bf16" else None
        codes = scales = None
        if format != "bf16":
            codes = torch.empty((M, H), dtype=torch.int8 if format == "int8" else torch.uint8, device=dev)
        if format == "fp8":
            scales = torch.empty((M, H // 128), dtype=torch.float32, device=dev)
        elif format == "mxfp8":
            scales = torch.empty((M, H // 32), dtype=torch.uint8, device=dev)
        elif format == "int8":
            scales = torch.empty((M,), dtype=torch.float32, device=dev)
        prob = api.norm_problem(
            M, H, format, eps, residual is not None and residual.dtype == torch.float32,
            weight.dtype == torch.float32, _row_stride(x),
            0 if residual is None else _row_stride(residual),
            0 if residual_out is None else _row_stride(residual_out))
        api.rmsnorm_quantize(prob, x, weight, residual_in=residual, residual_out=residual_out, norm_out=y,
                             codes=codes, scales=scales, static_scale=static_scale)
    return NormOutput(codes, scales, y, residual_out)


class Int8Linear:
    """A dense product in 8-bit integers on one GPU.

    weight:       int8 [N, K] (rows whose length is no multiple of 16 are
                  padded with zeros here, once)
    weight_scale: FP32 [N], one per channel
    bias:         FP32 [N] or None
    """

    def __init__(self, weight, weight_scale, bias=None):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise ValueError("weight: expected a tensor [N, K]")
        N, K = weight.shape
        _expect("weight", weight, (torch.int8,), (N, K))
        self.device = weight.device
        _expect("weight_scale", weight_scale, (torch.float32,), (N,), self.device)
        if bias is not None:
            _expect("bias", bias, (torch.float32,), (N,), self.device)
        self.out_features, self.in_features = N, K
        if _row_stride(weight, 16) % 16 or weight.data_ptr() % 16:
            padded = torch.zeros((N, -(-K // 16) * 16), dtype=torch.int8, device=self.device)
            padded[:, :K] = weight
            weight = padded[:, :K]
        self.weight, self.weight_scale, self.bias = weight, weight_scale, bias
        self._status = torch.zeros((1,), dtype=torch.int32, device=self.device)

    def forward(self, x, x_scale, out=None, out_dtype=torch.bfloat16, stream=None):
        """x int8 [M, K] (rows a multiple of 16 bytes apart), x_scale FP32 [M] -> out BF16 or FP32 [M, N]."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: expected a tensor [M, K]")
        M = x.shape[0]
        _expect("x", x, (torch.int8,), (M, self.in_features), self.device)
        _expect("x_scale", x_scale, (torch.float32,), (M,), self.device)
        if out is not None:
            _expect("out", out, (torch.bfloat16, torch.float32), (M, self.out_features), self.device)
        elif out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype {out_dtype}: expected torch.bfloat16 or torch.float32")
        with _on(self.device, stream):
            if out is None:
                out = torch.empty((M, self.out_features), dtype=out_dtype, device=self.device)
            prob = api.int8_problem(M, self.in_features, self.out_features, out.dtype == torch.float32,
                                    _row_stride(x, 16), _row_stride(self.weight, 16), _row_stride(out))
            api.matmul_int8(prob, x, x_scale, self.weight, self.weight_scale, out, self._status, bias=self.bias)
        return out

    def check_status(self):
        """Raise if a call on this object gave up a wait (synchronises)."""
        code = int(self._status.item())
        if code != api.MOE_OK:
            raise api.MoEError("device status", code)


class LayoutBuffers:
    """Caller-owned device arrays of ``moe_layout_t`` for one problem size."""

    def __init__(self, M, k, E, device):
        R = M * k
        self.expert_counts = _i32(E, device)
        self.expert_start_indices = _i32(E + 1, device)
        self.src_info = _i32(R, device)
        self.slot_to_row = _i32(R, device)
        self.expert_ids = _i32(E, device)
        self.num_active = _i32(1, device)
        self.a_scale_offsets = _i32(E + 1, device)
        self.tile_offsets = _i32(E + 1, device)
        self.struct = api.layout(self.expert_counts, self.expert_start_indices, self.src_info,
                                 self.slot_to_row, self.expert_ids, self.num_active,
                                 self.a_scale_offsets, self.tile_offsets)

    def host(self):
        return {k: getattr(self, k).cpu().numpy() for k in (
            "expert_counts", "expert_start_indices", "src_info", "slot_to_row", "expert_ids",
            "num_active", "a_scale_offsets", "tile_offsets")}


class MoELayer:
    """One routed-MoE FFN layer on one GPU.

    p:       problem dict (hidden, intermediate_hidden, num_experts, num_topk,
             activation_clamp, format, num_tokens = the largest batch served)
    weights: dict of device tensors w13, w13_scale, w2, w2_scale and, for
             NVFP4, gate_up_expert_scales, down_expert_scales, c_input_scales
             (FP8 per-tensor: c_input_scales) in the logical layouts of
             include/moe.h; the weights are prepared here
    p may also carry "shared_expert" (0/1), "activation" ("swiglu" |
    "swigluoai") and "activation_alpha"
    p may also carry "tile_regime" ("auto", "large_m", "small_m")
    """

    def __init__(self, p, weights, device=None, fast_math=1):
        self.p = dict(p)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.fast_math = fast_math
        api.init(self.device.index if self.device.index is not None else 0)
        self.max_tokens = int(p["num_tokens"])
        # a fused shared expert (p["shared_expert"] = 1) is one more expert
        # and one more slot per token after the routing
        self.shared = int(p.get("shared_expert", 0))
        self.k_all = int(p["num_topk"]) + self.shared
        self.E_all = int(p["num_experts"]) + self.shared
        self.prob = api.problem_from_dict(self.p, fast_math=fast_math)
        w = weights
        self.alpha1 = w.get("gate_up_expert_scales")
        self.alpha2 = w.get("down_expert_scales")
        self.c_in = w.get("c_input_scales")
        # FP8 block and per-tensor scales stay logical; NVFP4 and MXFP8 scales
        # go into the prepared blobs
        keep = self.p["format"] in ("fp8", "fp8_tensor")
        self.w13_scale = w.get("w13_scale") if keep else None
        self.w2_scale = w.get("w2_scale") if keep else None
        n13, n2 = api.prepared_weights_size(self.prob)
        self.w13 = torch.empty(n13, dtype=torch.uint8, device=self.device)
        self.w2 = torch.empty(n2, dtype=torch.uint8, device=self.device)
        logical = api.weights(w["w13"], w.get("w13_scale"), w["w2"], w.get("w2_scale"))
        api.prepare_weights(self.prob, logical, self.w13, self.w2)
        self.weights = api.weights(self.w13, self.w13_scale, self.w2, self.w2_scale,
                                   self.alpha1, self.alpha2, self.c_in)
        self.ws_bytes = api.workspace_size(self.prob)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        api.workspace_init(self.ws, self.ws_bytes)

    def problem(self, M):
        if M > self.max_tokens:
            raise ValueError(f"{M} tokens > the {self.max_tokens} this layer was sized for")
        return api.problem_from_dict(self.p, num_tokens=M, fast_math=self.fast_math)

    def forward(self, x, x_scale=None, topk_idx=None, topk_weights=None, logits=None, bias=None,
                out=None, stream=None, x_rowwise_scale=None):
        """moe_fused: the whole layer, BF16 out [M, H]."""
        M = x.shape[0]
        if out is None:
            out = torch.empty((M, self.p["hidden"]), dtype=torch.bfloat16, device=self.device)
        api.fused(self.problem(M), api.act(x, x_scale, x_rowwise_scale), self.weights, out, self.ws,
                  self.ws_bytes, topk_idx=topk_idx, topk_weights=topk_weights, logits=logits, bias=bias,
                  stream=stream)
        return out

    def quantize_rowwise(self, x_bf16, stream=None):
        """Per-token dynamic NVFP4 quantisation of BF16 activations [M, H]:
        (codes uint8 [M, H/2], block scales E4M3 [M, H/16], rowwise BF16 [M])."""
        M, H = x_bf16.shape
        codes = torch.empty((M, H // 2), dtype=torch.uint8, device=self.device)
        scales = torch.empty((M, H // 16), dtype=torch.uint8, device=self.device)
        rowwise = torch.empty((M,), dtype=torch.int16, device=self.device)
        api.quantize_nvfp4_rowwise(self.problem(M), x_bf16, codes, scales, rowwise, stream=stream)
        return codes, scales, rowwise

    def norm_quantize(self, x, weight, residual=None, eps=1e-6, x_scale=None, residual_out=None, stream=None):
        """Residual addition and RMS norm of x BF16 [M, H] into this layer's
        activation encoding: (activations, x_scale, x_rowwise_scale, normed
        BF16 [M, H], residual out), as forward takes them.  x_scale: FP8
        per-tensor layers' static scale, FP32 [1].  NVFP4 rows are quantised
        per token (gate_up_expert_scales hold the weights' scales alone)."""
        fmt = self.p["format"]
        _expect("x", x, (torch.bfloat16,), (x.shape[0], self.p["hidden"]), self.device)
        if (fmt == "fp8_tensor") != (x_scale is not None):
            raise ValueError("x_scale is the static scale of FP8 per-tensor activations, and of no others")
        n = rmsnorm_quantize(x, weight, residual, "bf16" if fmt == "nvfp4" else fmt, eps, x_scale, norm=True,
                             residual_out=residual_out, stream=stream)
        if fmt == "bf16":
            return n.norm, None, None, n.norm, n.residual
        if fmt == "nvfp4":
            with _on(self.device, stream):
                codes, scales, rowwise = self.quantize_rowwise(n.norm)
            return codes, scales, rowwise, n.norm, n.residual
        return n.codes, x_scale if fmt == "fp8_tensor" else n.scales, None, n.norm, n.residual

    def router_logits(self, x, router_weight, stream=None):
        """Router logits FP32 [M, E] of the normed rows x BF16 [M, H];
        router_weight BF16 [E, H]."""
        M, E, H = x.shape[0], self.p["num_experts"], self.p["hidden"]
        _expect("x", x, (torch.bfloat16,), (M, H), self.device)
        _expect("router_weight", router_weight, (torch.bfloat16,), (E, H), self.device)
        if not x.is_contiguous() or not router_weight.is_contiguous():
            raise ValueError("x and router_weight must be contiguous")
        with _on(self.device, stream):
            logits = torch.empty((M, E), dtype=torch.float32, device=self.device)
            api.router_logits(self.problem(M), x, router_weight, logits, self.ws)
        return logits

    def forward_prenorm(self, x, norm_weight, router_weight, residual=None, bias=None, eps=1e-6, x_scale=None,
                        residual_out=None, stream=None):
        """A pre-norm block's routed half: the residual's addition, the norm,
        the router and the layer.  x BF16 [M, H]; returns (layer output BF16
        [M, H], residual out: the stream the output is to be added to)."""
        with _on(self.device, stream):
            q, q_scale, rowwise, normed, res = self.norm_quantize(x, norm_weight, residual, eps, x_scale, residual_out)
            logits = self.router_logits(normed, router_weight)
            out = self.forward(q, q_scale, logits=logits, bias=bias, x_rowwise_scale=rowwise)
        return out, (x if residual is None else res)

    def shared_slots(self, topk_idx, topk_weights):
        """Precomputed routing [M, k] -> [M, k + 1]: the shared expert's slot
        (index num_experts, weight 1) appended, as every call after the
        routing expects when the layer has a shared expert."""
        if not self.shared:
            return topk_idx, topk_weights
        M = topk_idx.shape[0]
        idx = torch.cat([topk_idx, torch.full((M, 1), self.p["num_experts"], dtype=topk_idx.dtype,
                                              device=topk_idx.device)], dim=1)
        w = torch.cat([topk_weights, torch.ones((M, 1), dtype=topk_weights.dtype, device=topk_weights.device)],
                      dim=1)
        return idx.contiguous(), w.contiguous()

    def route(self, logits, bias=None, stream=None):
        M = logits.shape[0]
        k = self.k_all
        idx = torch.empty((M, k), dtype=torch.int64, device=self.device)
        w = torch.empty((M, k), dtype=torch.float32, device=self.device)
        api.route(self.problem(M), logits, bias, idx, w, stream=stream)
        return idx, w

    def permute(self, topk_idx, stream=None):
        M = topk_idx.shape[0]
        lay = LayoutBuffers(M, self.k_all, self.E_all, self.device)
        api.permute(self.problem(M), topk_idx, lay.struct, self.ws, self.ws_bytes, stream=stream)
        return lay

    def ffn(self, x, x_scale, lay, topk_weights, out_mode=api.MOE_OUT_ACCUMULATE, keep_intermediate=False,
            stream=None, x_rowwise_scale=None):
        """moe_ffn; returns (out fp32, intermediate bytes or None)."""
        M = x.shape[0]
        prob = self.problem(M)
        H = self.p["hidden"]
        rows = M if out_mode == api.MOE_OUT_ACCUMULATE else M * self.k_all
        out = torch.empty((rows, H), dtype=torch.float32, device=self.device)
        inter = None
        if keep_intermediate:
            n, _ = api.intermediate_size(prob)
            inter = torch.empty(n, dtype=torch.uint8, device=self.device)
        api.ffn(prob, api.act(x, x_scale, x_rowwise_scale), self.weights, lay.struct, topk_weights, out_mode, out,
                self.ws, self.ws_bytes, intermediate=inter, stream=stream)
        return out, inter

    def combine(self, lay, topk_weights, inp, in_mode, M, stream=None):
        out = torch.empty((M, self.p["hidden"]), dtype=torch.bfloat16, device=self.device)
        api.combine(self.problem(M), lay.struct if lay is not None else None, topk_weights, inp, in_mode,
                    out, stream=stream)
        return out

    def workspace_views(self, M):
        """Device views of what the last moe_fused call with M tokens left in
        the workspace (layout arrays, in-kernel routing, the re-quantised
        intermediate and its scales, the FP32 accumulator), for inspection.
        Read them only after that call has completed."""
        prob = self.problem(M)
        off = api.workspace_offsets(prob)
        k, E, H = self.k_all, self.E_all, self.p["hidden"]
        R = M * k
        n_int, so = api.intermediate_size(prob)
        ws = self.ws

        def i32(name, n):
            return ws[off[name]: off[name] + 4 * n].view(torch.int32)

        v = {name: i32(name, n) for name, n in (
            ("expert_counts", E), ("expert_start_indices", E + 1), ("src_info", R), ("slot_to_row", R),
            ("expert_ids", E), ("num_active", 1), ("a_scale_offsets", E + 1), ("tile_offsets", E + 1))}
        v["topk_idx"] = ws[off["topk_idx"]: off["topk_idx"] + 8 * R].view(torch.int64).view(M, k)
        v["topk_weights"] = ws[off["topk_weights"]: off["topk_weights"] + 4 * R].view(torch.float32).view(M, k)
        v["intermediate"] = ws[off["intermediate"]: off["intermediate"] + so]
        v["intermediate_scales"] = ws[off["intermediate_scales"]: off["intermediate_scales"] + (n_int - so)]
        v["scale_rows"] = off["scale_rows"]
        v["accumulator"] = ws[off["accumulator"]: off["accumulator"] + 4 * M * H].view(torch.float32).view(M, H)
        return v

    def status(self, stream=None):
        return api.read_status(self.ws, stream=stream)

    def check_status(self, stream=None):
        code = self.status(stream)
        if code != api.MOE_OK:
            raise api.MoEError("device status", code)

    def clear_status(self, stream=None):
        api.workspace_init(self.ws, self.ws_bytes, stream=stream)
