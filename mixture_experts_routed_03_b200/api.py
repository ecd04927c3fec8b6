"""ctypes binding of ``include/moe.h`` (``libmoe_b200.so``).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Tensor arguments may be torch tensors (their ``data_ptr()``
is passed), plain integers (raw device addresses) or ``None`` (NULL).
Streams are torch streams, raw ``cudaStream_t`` integers, or ``None`` for
torch's current stream.

The library is loaded on first use from this package directory; a missing
library raises ``RuntimeError`` -- there is no fallback of any kind.
"""

import ctypes
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libmoe_b200.so"
LIB_PATH = os.path.join(_HERE, LIB_NAME)

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_BAD_INDEX = 5
MOE_ERR_TIMEOUT = 6

FORMATS = {"bf16": 0, "fp8": 1, "nvfp4": 2, "mxfp8": 3, "fp8_tensor": 4}

MOE_OUT_ACCUMULATE = 0
MOE_OUT_STAGED = 1
MOE_IN_ACCUMULATED = 0
MOE_IN_STAGED = 1

# Every entry point declared in include/moe.h.
EXPORTS = (
    "moe_init", "moe_get_workspace_size", "moe_workspace_init", "moe_prepare_weights",
    "moe_get_prepared_weights_size",
    "moe_route", "moe_permute", "moe_ffn", "moe_get_intermediate_size", "moe_combine",
    "moe_fused", "moe_read_status", "moe_status_string", "moe_timing_enable", "moe_timing_read",
    "moe_permute_noalloc", "moe_get_tile_regime", "moe_get_workspace_offsets",
    "moe_workspace_test_hooks", "moe_quantize_nvfp4_rowwise",
    "moe_rmsnorm_quantize", "moe_router_logits", "moe_matmul_int8", "moe_get_product_plan",
    "moe_product_test_hooks",
)

SLOTS = ("route", "permute", "gather", "gemm1", "zero", "gemm2", "finalize", "combine", "fused")


class MoEError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn} returned {status_string(code)} ({code})")


class Problem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("intermediate_hidden", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("activation_clamp", ctypes.c_float),
        ("format", ctypes.c_int32),
        ("fast_math", ctypes.c_int32),
        ("tile_regime", ctypes.c_int32),
        ("shared_expert", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("activation_alpha", ctypes.c_float),
    ]


class Act(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_scale", ctypes.c_void_p), ("x_rowwise_scale", ctypes.c_void_p)]


class Weights(ctypes.Structure):
    _fields_ = [
        ("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
        ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
        ("gate_up_expert_scales", ctypes.c_void_p),
        ("down_expert_scales", ctypes.c_void_p),
        ("c_input_scales", ctypes.c_void_p),
    ]


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "expert_counts", "expert_start_indices", "src_info", "slot_to_row",
        "expert_ids", "num_active", "a_scale_offsets", "tile_offsets")]


class NormProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("residual_in_stride", ctypes.c_int64),
        ("residual_out_stride", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("residual_fp32", ctypes.c_int32),
        ("weight_fp32", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class Int8Problem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("w_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("out_fp32", ctypes.c_int32),
    ]


class ProductPlan(ctypes.Structure):
    _fields_ = [
        ("kernel", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("splits", ctypes.c_int32),
        ("stage_blocks", ctypes.c_int32),
        ("estimate_us", ctypes.c_float),
    ]


WS_OFFSET_FIELDS = ("status", "topk_idx", "topk_weights", "expert_counts", "expert_start_indices",
                    "src_info", "slot_to_row", "expert_ids", "num_active", "a_scale_offsets",
                    "tile_offsets", "intermediate", "intermediate_scales", "scale_rows", "accumulator")


class WorkspaceOffsets(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64 if n == "scale_rows" else ctypes.c_size_t) for n in WS_OFFSET_FIELDS]


_lib = None
_call = None      # the extension's call(address, *args)
_address = {}     # entry point -> address, for it


def _short(name):
    """(call, address) of an entry point that is called through the extension
    of csrc/binding.c: ctypes marshals ten arguments in two microseconds, as
    long as the kernels of a few tokens take.  Where the extension was not
    built, ctypes makes the same calls."""
    global _call
    if _call is None:
        L = lib()
        try:
            from ._binding import call
        except ImportError:
            call = _ctypes_call
        for n in ("moe_rmsnorm_quantize", "moe_router_logits", "moe_matmul_int8"):
            _address[n] = ctypes.cast(getattr(L, n), ctypes.c_void_p).value
        _call = call
    return _call, _address[name]


def _ctypes_call(address, *args):
    """csrc/binding.c's call(address, *args), by ctypes."""
    if len(args) not in (6, 9, 10):
        raise TypeError("call() makes calls of 6, 9 or 10 arguments")
    fn = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * len(args))(address)
    return fn(*[a if a is None or isinstance(a, int) else a.data_ptr() for a in args])


def lib():
    """The loaded library (loads it on first call; raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                               "(or python -m mixture_experts_routed_03_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER(Problem)
        sig = {
            "moe_init": [ctypes.c_int],
            "moe_get_workspace_size": [P, ctypes.POINTER(sz)],
            "moe_workspace_init": [vp, sz, vp],
            "moe_workspace_test_hooks": [vp, sz, i32, i32, vp],
            "moe_quantize_nvfp4_rowwise": [P, vp, vp, vp, vp, vp],
            "moe_rmsnorm_quantize": [ctypes.POINTER(NormProblem)] + [vp] * 9,
            "moe_router_logits": [P, vp, vp, vp, vp, vp],
            "moe_matmul_int8": [ctypes.POINTER(Int8Problem)] + [vp] * 8,
            "moe_get_product_plan": [i32, ctypes.c_int64, i32, i32, ctypes.POINTER(ProductPlan)],
            "moe_product_test_hooks": [i32, i32],
            "moe_prepare_weights": [P, ctypes.POINTER(Weights), vp, vp, vp],
            "moe_get_prepared_weights_size": [P, ctypes.POINTER(sz), ctypes.POINTER(sz)],
            "moe_route": [P, vp, vp, vp, vp, vp],
            "moe_permute": [P, vp, ctypes.POINTER(Layout), vp, sz, vp],
            "moe_ffn": [P, ctypes.POINTER(Act), ctypes.POINTER(Weights), ctypes.POINTER(Layout),
                        vp, i32, vp, vp, vp, sz, vp],
            "moe_get_intermediate_size": [P, ctypes.POINTER(sz), ctypes.POINTER(sz)],
            "moe_get_tile_regime": [P, ctypes.POINTER(i32)],
            "moe_get_workspace_offsets": [P, ctypes.POINTER(WorkspaceOffsets)],
            "moe_combine": [P, ctypes.POINTER(Layout), vp, vp, i32, vp, vp],
            "moe_fused": [P, ctypes.POINTER(Act), ctypes.POINTER(Weights), vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_read_status": [vp, vp],
            "moe_timing_enable": [ctypes.c_int, ctypes.c_int],
            "moe_permute_noalloc": [P, vp, ctypes.POINTER(Layout), vp, vp],
            "moe_timing_read": [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(code):
    try:
        return lib().moe_status_string(int(code)).decode()
    except RuntimeError:
        return str(code)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        import torch
        # the raw handle alone, where this torch gives it: a Stream object costs a microsecond a call
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _expect_struct(prob, cls):
    if type(prob) is not cls:
        raise TypeError(f"expected a {cls.__name__}, got {type(prob).__name__}")


def _check(fn, code):
    if code != MOE_OK:
        raise MoEError(fn, code)


TILE_REGIMES = {"auto": 0, "large_m": 1, "small_m": 2}
ACTIVATIONS = {"swiglu": 0, "swigluoai": 1}
PRODUCT_KERNELS = ("few", "warps", "tiles", "pairs")
PRODUCT_HOLDS = {"nothing": 0, "load": 1, "sum": 2, "load_of_second": 3}
NORM_FORMATS = {"bf16": 0, "fp8": 1, "mxfp8": 3, "fp8_tensor": 4, "int8": 5}


def problem(num_tokens, hidden, intermediate_hidden, num_experts, num_topk,
            activation_clamp=10.0, format="bf16", fast_math=1, tile_regime="auto", shared_expert=0,
            activation="swiglu", activation_alpha=1.702):
    """A moe_problem_t.  format: a FORMATS name or code; tile_regime: a
    TILE_REGIMES name or code; shared_expert: 0 or 1 (a fused shared expert,
    one more expert and slot after the routing); activation: "swiglu" or
    "swigluoai", whose gate slope is activation_alpha (1.702 by default, one
    public model's value; the pages leave it to the caller)."""
    fmt = FORMATS[format] if isinstance(format, str) else int(format)
    clamp = float(activation_clamp)
    regime = TILE_REGIMES[tile_regime] if isinstance(tile_regime, str) else int(tile_regime)
    act = ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)
    return Problem(int(num_tokens), int(hidden), int(intermediate_hidden), int(num_experts),
                   int(num_topk), math.inf if math.isinf(clamp) else clamp, fmt, int(fast_math), regime,
                   int(shared_expert), act, float(activation_alpha))


def problem_from_dict(d, num_tokens=None, fast_math=1):
    return problem(d["num_tokens"] if num_tokens is None else num_tokens, d["hidden"],
                   d["intermediate_hidden"], d["num_experts"], d["num_topk"],
                   d.get("activation_clamp", 10.0), d["format"], fast_math, d.get("tile_regime", "auto"),
                   d.get("shared_expert", 0), d.get("activation", "swiglu"), d.get("activation_alpha", 1.702))


def norm_problem(num_tokens, hidden, format="bf16", eps=1e-6, residual_fp32=False, weight_fp32=False, x_stride=0,
                 residual_in_stride=0, residual_out_stride=0):
    """A moe_norm_t.  format: a NORM_FORMATS name or code; strides in
    elements, 0 meaning hidden."""
    fmt = NORM_FORMATS[format] if isinstance(format, str) else int(format)
    return NormProblem(int(num_tokens), int(x_stride), int(residual_in_stride), int(residual_out_stride),
                       int(hidden), fmt, int(residual_fp32), int(weight_fp32), float(eps))


def int8_problem(num_tokens, in_features, out_features, out_fp32=False, x_stride=0, w_stride=0, out_stride=0):
    """A moe_int8_matmul_t; strides in elements, 0 meaning the row's length."""
    return Int8Problem(int(num_tokens), int(x_stride), int(w_stride), int(out_stride), int(in_features),
                       int(out_features), int(out_fp32))


def act(x, x_scale=None, x_rowwise_scale=None):
    return Act(_ptr(x), _ptr(x_scale), _ptr(x_rowwise_scale))


def weights(w13, w13_scale, w2, w2_scale, gate_up_expert_scales=None, down_expert_scales=None,
            c_input_scales=None):
    return Weights(_ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                   _ptr(gate_up_expert_scales), _ptr(down_expert_scales), _ptr(c_input_scales))


def layout(expert_counts, expert_start_indices, src_info, slot_to_row, expert_ids, num_active,
           a_scale_offsets, tile_offsets):
    return Layout(*(_ptr(t) for t in (expert_counts, expert_start_indices, src_info, slot_to_row,
                                      expert_ids, num_active, a_scale_offsets, tile_offsets)))


# ---------------------------------------------------------------- entry points

def init(device=0):
    _check("moe_init", lib().moe_init(int(device)))


def workspace_size(prob):
    n = ctypes.c_size_t(0)
    _check("moe_get_workspace_size", lib().moe_get_workspace_size(ctypes.byref(prob), ctypes.byref(n)))
    return n.value


def tile_regime(prob):
    """'large_m' or 'small_m': the grouped GEMMs' tile shape for this problem."""
    r = ctypes.c_int32(0)
    _check("moe_get_tile_regime", lib().moe_get_tile_regime(ctypes.byref(prob), ctypes.byref(r)))
    return {v: k for k, v in TILE_REGIMES.items()}[r.value]


def workspace_offsets(prob):
    """{region: byte offset} of moe_fused's working data in the workspace
    (plus 'scale_rows', the padded scale rows P)."""
    o = WorkspaceOffsets()
    _check("moe_get_workspace_offsets", lib().moe_get_workspace_offsets(ctypes.byref(prob), ctypes.byref(o)))
    return {n: int(getattr(o, n)) for n in WS_OFFSET_FIELDS}


def intermediate_size(prob):
    n, off = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_get_intermediate_size",
           lib().moe_get_intermediate_size(ctypes.byref(prob), ctypes.byref(n), ctypes.byref(off)))
    return n.value, off.value


def workspace_init(ws, nbytes, stream=None):
    _check("moe_workspace_init", lib().moe_workspace_init(_ptr(ws), int(nbytes), _stream(stream)))


def workspace_test_hooks(ws, nbytes, wait_limit_us=0, skip_arrival=0, stream=None):
    """Failure-detection test hooks in the workspace header (see include/moe.h)."""
    _check("moe_workspace_test_hooks", lib().moe_workspace_test_hooks(_ptr(ws), int(nbytes), int(wait_limit_us),
                                                                      int(skip_arrival), _stream(stream)))


def prepared_weights_size(prob):
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_get_prepared_weights_size",
           lib().moe_get_prepared_weights_size(ctypes.byref(prob), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def prepare_weights(prob, logical, out_w13, out_w2, stream=None):
    _check("moe_prepare_weights", lib().moe_prepare_weights(
        ctypes.byref(prob), ctypes.byref(logical), _ptr(out_w13), _ptr(out_w2), _stream(stream)))


def route(prob, logits, bias, topk_idx, topk_weights, stream=None):
    _check("moe_route", lib().moe_route(ctypes.byref(prob), _ptr(logits), _ptr(bias), _ptr(topk_idx),
                                        _ptr(topk_weights), _stream(stream)))


def quantize_nvfp4_rowwise(prob, x_bf16, codes, block_scales, rowwise_scales, stream=None):
    """Per-token dynamic NVFP4 quantisation of BF16 activations (see include/moe.h)."""
    _check("moe_quantize_nvfp4_rowwise", lib().moe_quantize_nvfp4_rowwise(
        ctypes.byref(prob), _ptr(x_bf16), _ptr(codes), _ptr(block_scales), _ptr(rowwise_scales), _stream(stream)))


def rmsnorm_quantize(prob, x, weight, residual_in=None, residual_out=None, norm_out=None, codes=None, scales=None,
                     static_scale=None, stream=None):
    """Residual addition, RMS norm and activation encoding in one pass (see
    include/moe.h); prob: a NormProblem."""
    _expect_struct(prob, NormProblem)
    call, at = _short("moe_rmsnorm_quantize")
    code = call(at, ctypes.addressof(prob), x, residual_in, weight, static_scale, residual_out, norm_out, codes, scales,
                _stream(stream))
    if code:
        raise MoEError("moe_rmsnorm_quantize", code)


def router_logits(prob, x_bf16, router_weight, logits, device_status, stream=None):
    """Router logits fp32 [M, E] of BF16 rows (see include/moe.h); prob: the
    layer's Problem, device_status: an int32 on the device (or a workspace)."""
    _expect_struct(prob, Problem)
    call, at = _short("moe_router_logits")
    code = call(at, ctypes.addressof(prob), x_bf16, router_weight, logits, device_status, _stream(stream))
    if code:
        raise MoEError("moe_router_logits", code)


def matmul_int8(prob, x, x_scale, w, w_scale, out, device_status, bias=None, stream=None):
    """Product of 8-bit integers with a scale per token and per channel (see
    include/moe.h); prob: an Int8Problem."""
    _expect_struct(prob, Int8Problem)
    call, at = _short("moe_matmul_int8")
    code = call(at, ctypes.addressof(prob), x, x_scale, w, w_scale, bias, out, device_status, _stream(stream))
    if code:
        raise MoEError("moe_matmul_int8", code)


def product_plan(is_int8, num_tokens, in_features, out_features):
    """The ProductPlan of matmul_int8 or router_logits at these sizes (host
    only); its kernel is a PRODUCT_KERNELS index."""
    plan = ProductPlan()
    _check("moe_get_product_plan", lib().moe_get_product_plan(int(bool(is_int8)), int(num_tokens), int(in_features),
                                                              int(out_features), ctypes.byref(plan)))
    return plan


def product_test_hooks(wait_limit_us=0, hold="nothing"):
    """Test hook of the products' failure detection: a wait limit and an event
    that never comes, for calls from now on (see include/moe.h); no arguments
    end it.  hold: a PRODUCT_HOLDS name or code."""
    code = PRODUCT_HOLDS[hold] if isinstance(hold, str) else int(hold)
    _check("moe_product_test_hooks", lib().moe_product_test_hooks(int(wait_limit_us), code))


def permute(prob, topk_idx, lay, ws, ws_bytes, stream=None):
    _check("moe_permute", lib().moe_permute(ctypes.byref(prob), _ptr(topk_idx), ctypes.byref(lay),
                                            _ptr(ws), int(ws_bytes), _stream(stream)))


def ffn(prob, a, w, lay, topk_weights, out_mode, out, ws, ws_bytes, intermediate=None, stream=None):
    _check("moe_ffn", lib().moe_ffn(ctypes.byref(prob), ctypes.byref(a), ctypes.byref(w),
                                    ctypes.byref(lay), _ptr(topk_weights), int(out_mode), _ptr(out),
                                    _ptr(intermediate), _ptr(ws), int(ws_bytes), _stream(stream)))


def combine(prob, lay, topk_weights, inp, in_mode, out_bf16, stream=None):
    _check("moe_combine", lib().moe_combine(ctypes.byref(prob), None if lay is None else ctypes.byref(lay),
                                            _ptr(topk_weights), _ptr(inp), int(in_mode),
                                            _ptr(out_bf16), _stream(stream)))


def permute_noalloc(prob, topk_idx, lay, device_status, stream=None):
    """moe_permute without a workspace (see include/moe.h)."""
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(ctypes.byref(prob), _ptr(topk_idx),
                                                            ctypes.byref(lay), _ptr(device_status),
                                                            _stream(stream)))


def fused(prob, a, w, out_bf16, ws, ws_bytes, topk_idx=None, topk_weights=None, logits=None,
          bias=None, stream=None):
    _check("moe_fused", lib().moe_fused(ctypes.byref(prob), ctypes.byref(a), ctypes.byref(w),
                                        _ptr(topk_idx), _ptr(topk_weights), _ptr(logits), _ptr(bias),
                                        _ptr(out_bf16), _ptr(ws), int(ws_bytes), _stream(stream)))


def read_status(ws, stream=None):
    """Synchronise the stream and return the sticky device status code."""
    return lib().moe_read_status(_ptr(ws), _stream(stream))


def timing_enable(enable=True, max_calls=1024):
    _check("moe_timing_enable", lib().moe_timing_enable(int(bool(enable)), int(max_calls)))


def timing_read():
    """{slot: (summed ms, launches)} since the last read (waits for the events)."""
    ms = (ctypes.c_float * len(SLOTS))()
    n = (ctypes.c_int * len(SLOTS))()
    _check("moe_timing_read", lib().moe_timing_read(ms, n))
    return {name: (float(ms[i]), int(n[i])) for i, name in enumerate(SLOTS)}


def raw(fn_name, *args):
    """Call an entry point with raw ctypes arguments and return its status code."""
    return getattr(lib(), fn_name)(*args)
