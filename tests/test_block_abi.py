"""Argument checks of the operators next to the layer: refused on the host,
before anything is launched (the pointers are never dereferenced).  CPU only."""

import ctypes
import importlib.machinery
import os
import shutil
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from mixture_experts_routed_03_b200 import api, build, layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUPPORTED, OK = api.MOE_ERR_INVALID_ARG, api.MOE_ERR_UNSUPPORTED, api.MOE_OK
AT = 1 << 30          # made-up addresses, far apart


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


def _at(i, offset=0):
    return AT * (i + 1) + offset


# ------------------------------------------------------------------ struct layout

def test_struct_layouts_match_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"moe_norm_t": api.NormProblem, "moe_int8_matmul_t": api.Int8Problem}
    body = "".join(f'printf("{n} size %zu\\n", sizeof({n}));' +
                   "".join(f'printf("{n} {f} %zu\\n", offsetof({n}, {f}));' for f, _ in c._fields_)
                   for n, c in structs.items())
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {' + body + "return 0;}\n")
    exe = tmp_path / "l"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    table = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for n, c in structs.items():
        assert ctypes.sizeof(c) == table[(n, "size")]
        for f, _ in c._fields_:
            assert getattr(c, f).offset == table[(n, f)], (n, f)


# ------------------------------------------------------------------ norm

def _norm(lib, problem=None, **kw):
    p = problem if problem is not None else api.norm_problem(4, 256, "fp8")
    a = dict(x=_at(0), residual_in=_at(1), weight=_at(2), static_scale=None, residual_out=_at(3), norm_out=_at(4),
             codes=_at(5), scales=_at(6))
    a.update(kw)
    return lib.moe_rmsnorm_quantize(ctypes.byref(p), a["x"], a["residual_in"], a["weight"], a["static_scale"],
                                    a["residual_out"], a["norm_out"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), BAD), (dict(hidden=0), BAD), (dict(hidden=128), BAD), (dict(hidden=300), BAD),
    (dict(hidden=32768 + 256), UNSUPPORTED), (dict(num_tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(format=2), BAD), (dict(format=6), BAD), (dict(format=-1), BAD),
    (dict(eps=0.0), BAD), (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(residual_fp32=2), BAD), (dict(weight_fp32=-1), BAD),
    (dict(x_stride=248), BAD), (dict(x_stride=260), BAD), (dict(x_stride=-256), BAD),
    (dict(residual_in_stride=252), BAD), (dict(residual_out_stride=260), BAD),
    (dict(residual_out_stride=258, residual_fp32=1), BAD), (dict(x_stride=(1 << 31) + 8), BAD),
])
def test_norm_problem_refused(lib, kw, code):
    d = dict(num_tokens=4, hidden=256, format="fp8")
    d.update(kw)
    assert _norm(lib, api.norm_problem(**d)) == code


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(weight=None), dict(codes=None), dict(scales=None), dict(residual_in=None),
    dict(x=_at(0, 8)), dict(weight=_at(2, 4)), dict(residual_in=_at(1, 8)), dict(residual_out=_at(3, 2)),
    dict(norm_out=_at(4, 8)), dict(codes=_at(5, 8)), dict(scales=_at(6, 2)), dict(static_scale=_at(7)),
    dict(norm_out=_at(0)),                               # over the input
    dict(codes=_at(1, 1024)),                            # inside the residual
    dict(codes=_at(4, 2032)),                            # over the last row of another output
    dict(residual_out=_at(1, 512)),                      # shifted by a row: not in place
    dict(scales=_at(2, 256)),                            # over the weight
])
def test_norm_arguments_refused(lib, kw):
    assert _norm(lib, **kw) == BAD


def test_norm_format_arguments(lib):
    bf16 = api.norm_problem(4, 256, "bf16")
    assert _norm(lib, bf16, codes=None, scales=None, norm_out=None) == BAD
    assert _norm(lib, bf16, scales=None) == BAD
    assert _norm(lib, bf16, codes=None) == BAD
    tensor = api.norm_problem(4, 256, "fp8_tensor")
    assert _norm(lib, tensor) == BAD                     # no static scale
    assert _norm(lib, tensor, static_scale=_at(7)) == BAD                    # scales are not written
    assert _norm(lib, tensor, static_scale=_at(7, 2), scales=None) == BAD
    # in place only with one stride
    p = api.norm_problem(4, 256, "fp8", residual_in_stride=256, residual_out_stride=512)
    assert _norm(lib, p, residual_out=_at(1)) == BAD


def test_norm_of_no_tokens_is_ok(lib):
    p = api.norm_problem(0, 256, "int8")
    assert lib.moe_rmsnorm_quantize(ctypes.byref(p), *([None] * 9)) == OK
    assert lib.moe_rmsnorm_quantize(None, *([None] * 9)) == BAD


# ------------------------------------------------------------------ router

def test_router_arguments_refused(lib):
    p = api.problem(4, 256, 128, 8, 2)

    def call(x=_at(0), w=_at(1), logits=_at(2), status=_at(3), prob=p):
        return lib.moe_router_logits(ctypes.byref(prob), x, w, logits, status, None)

    for kw in (dict(x=None), dict(w=None), dict(logits=None), dict(status=None), dict(x=_at(0, 8)),
               dict(w=_at(1, 8)), dict(logits=_at(2, 2)), dict(status=_at(3, 1)), dict(logits=_at(0, 64)),
               dict(logits=_at(1, 4096 - 16)), dict(status=_at(2, 124))):
        assert call(**kw) == BAD, kw
    assert call(prob=api.problem(4, 300, 128, 8, 2)) == BAD
    assert call(prob=api.problem(4, 256, 128, 2000, 2)) == UNSUPPORTED
    assert call(prob=api.problem(4, (1 << 29) + 256, 128, 1, 1)) == UNSUPPORTED
    assert call(prob=api.problem(0, 256, 128, 8, 2), x=None, w=None, logits=None, status=None) == OK


# ------------------------------------------------------------------ 8-bit integers

def _int8(lib, problem=None, **kw):
    p = problem if problem is not None else api.int8_problem(4, 64, 8)
    a = dict(x=_at(0), x_scale=_at(1), w=_at(2), w_scale=_at(3), bias=_at(4), out=_at(5), status=_at(6))
    a.update(kw)
    return lib.moe_matmul_int8(ctypes.byref(p), a["x"], a["x_scale"], a["w"], a["w_scale"], a["bias"], a["out"],
                               a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), BAD), (dict(in_features=0), BAD), (dict(out_features=0), BAD), (dict(out_fp32=2), BAD),
    (dict(in_features=65), BAD),                         # rows of 65 bytes cannot be loaded: pad them
    (dict(x_stride=48), BAD), (dict(x_stride=72), BAD), (dict(w_stride=63), BAD), (dict(out_stride=7), BAD),
    (dict(x_stride=-64), BAD), (dict(x_stride=(1 << 31) + 16), BAD), (dict(out_stride=(1 << 31) + 1), BAD),
    (dict(in_features=131072), UNSUPPORTED), (dict(num_tokens=(1 << 30) + 1), UNSUPPORTED),
])
def test_int8_problem_refused(lib, kw, code):
    d = dict(num_tokens=4, in_features=64, out_features=8)
    d.update(kw)
    assert _int8(lib, api.int8_problem(**d)) == code


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x_scale=None), dict(w=None), dict(w_scale=None), dict(out=None), dict(status=None),
    dict(x=_at(0, 8)), dict(w=_at(2, 4)), dict(x_scale=_at(1, 2)), dict(w_scale=_at(3, 1)), dict(bias=_at(4, 2)),
    dict(out=_at(5, 1)), dict(status=_at(6, 2)),
    dict(out=_at(0, 128)), dict(out=_at(2, 510)), dict(out=_at(1)), dict(out=_at(3, 28)), dict(out=_at(4)),
    dict(status=_at(5, 60)),
])
def test_int8_arguments_refused(lib, kw):
    assert _int8(lib, **kw) == BAD


def test_int8_of_no_tokens_is_ok(lib):
    p = api.int8_problem(0, 64, 8)
    assert lib.moe_matmul_int8(ctypes.byref(p), *([None] * 8)) == OK


# ------------------------------------------------------------------ the Python objects' own checks

def test_python_checks_raise_before_any_call():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = torch.zeros((256,), dtype=torch.bfloat16)
    for args, kw in (((x.float(), w), {}), ((x, w[:128]), {}), ((x, w.to(torch.float16)), {}),
                     ((x[0], w), {}), ((x.t(), w), {}), ((x, w), dict(residual=x[:2])),
                     ((x, w), dict(residual_out=x)), ((x, w), dict(residual=x.double())),
                     ((x, w), dict(format="nvfp4")), ((x, w), dict(static_scale=w[:1])),
                     (([1.0], w), {}), ((x[:1].expand(4, 256), w), {}),
                     ((x, w), dict(residual=x[:1].expand(4, 256))),
                     ((x, w), dict(residual=x, residual_out=x[:1].expand(4, 256)))):
        with pytest.raises(ValueError):
            layer.rmsnorm_quantize(*args, **kw)
    i = torch.zeros((8, 64), dtype=torch.int8)
    s = torch.zeros((8,), dtype=torch.float32)
    for args in ((i.float(), s), (i, s[:4]), (i[0], s), (i, s.double()), (i, s, s[:4]), (i.t(), s)):
        with pytest.raises(ValueError):
            layer.Int8Linear(*args)
    lin = layer.Int8Linear(i, s)
    for args, kw in (((i[:1].expand(8, 64), s), {}), ((i[:, :32], s), {}), ((i, s[:4]), {}), ((i[0], s), {}), ((i.float(), s), {}),
                     ((i, s), dict(out_dtype=torch.float16)), ((i, s), dict(out=torch.zeros((8, 7))))):
        with pytest.raises(ValueError):
            lin.forward(*args, **kw)


def test_int8_linear_pads_odd_rows_once():
    w = torch.arange(-64, 66, dtype=torch.int8).view(10, 13)
    lin = layer.Int8Linear(w, torch.ones(10))
    assert lin.weight.shape == (10, 13) and lin.weight.stride() == (16, 1)
    assert torch.equal(lin.weight, w)
    kept = torch.zeros((4, 32), dtype=torch.int8)
    assert layer.Int8Linear(kept, torch.ones(4)).weight.data_ptr() == kept.data_ptr()


# ------------------------------------------------------------------ the binding of the short calls

def test_binding_takes_tensors_integers_and_none(lib):
    x = torch.zeros(16)
    api.rmsnorm_quantize(api.norm_problem(0, 256, "int8"), None, x, codes=_at(0), stream=0)
    api.router_logits(api.problem(0, 256, 128, 8, 2), x, None, _at(0), x, stream=0)
    api.matmul_int8(api.int8_problem(0, 64, 8), x, x, None, _at(1), x, x, stream=0)


def test_binding_raises_the_librarys_errors(lib):
    for call in (lambda: api.rmsnorm_quantize(api.norm_problem(4, 100, "fp8"), None, None, stream=0),
                 lambda: api.router_logits(api.problem(4, 256, 128, 8, 2), _at(0, 8), _at(1), _at(2), _at(3), stream=0),
                 lambda: api.matmul_int8(api.int8_problem(4, 64, 8), _at(0), _at(1), _at(2), _at(3), _at(5, 1), _at(6),
                                         stream=0)):
        with pytest.raises(api.MoEError) as e:
            call()
        assert e.value.code == BAD and "MOE_ERR_INVALID_ARG" in str(e.value)


def test_binding_refuses_what_is_no_problem_or_pointer(lib):
    with pytest.raises(TypeError):
        api.rmsnorm_quantize(api.int8_problem(4, 64, 8), None, None, stream=0)
    with pytest.raises(TypeError):
        api.matmul_int8(api.norm_problem(4, 256), None, None, None, None, None, None, stream=0)
    with pytest.raises(TypeError):
        api.router_logits(None, None, None, None, None, stream=0)
    with pytest.raises(AttributeError):
        api.router_logits(api.problem(4, 256, 128, 8, 2), "x", None, None, None, stream=0)


def test_binding_function_checks_its_own_arguments(lib):
    call, at = api._short("moe_router_logits")
    for args in ((), (at,), (at, 0), (at,) + (0,) * 13):
        with pytest.raises(TypeError):
            call(*args)


# ------------------------------------------------------------------ without the extension

@pytest.fixture
def without_extension(lib, monkeypatch):
    """api as it is where csrc/binding.c was not built."""
    monkeypatch.setitem(sys.modules, "mixture_experts_routed_03_b200._binding", None)
    monkeypatch.setattr(api, "_call", None)
    assert api._short("moe_router_logits")[0] is api._ctypes_call


def test_calls_without_the_extension(without_extension, lib):
    test_binding_takes_tensors_integers_and_none(lib)
    test_binding_raises_the_librarys_errors(lib)
    test_binding_refuses_what_is_no_problem_or_pointer(lib)
    test_binding_function_checks_its_own_arguments(lib)


def test_extension_bears_the_interpreters_tag_and_is_the_one_loaded(lib):
    from mixture_experts_routed_03_b200 import _binding
    assert os.path.basename(build.BINDING_OUT) == "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0]
    assert _binding.__file__ == build.BINDING_OUT


@pytest.mark.parametrize("cc", ["missing", "failing"])
def test_build_without_a_c_compiler_or_python_headers_warns(cc, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BINDING_OUT", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build.shutil, "which", lambda name: None if cc == "missing" else "false")
    (tmp_path / "_binding.so").write_text("built from an older source")
    with pytest.warns(UserWarning, match="not built"):
        build._build_binding()
    assert not (tmp_path / "_binding.so").exists()       # nothing stale is left to be loaded


@pytest.mark.parametrize("private", [True, False])
def test_current_stream_with_and_without_torchs_private_call(private, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=42))
    if private:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 40 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert api._stream(None) == (43 if private else 42)
    assert api._stream(7) == 7 and api._stream(SimpleNamespace(cuda_stream=8)) == 8


# ------------------------------------------------------------------ the products' test hook

def test_product_test_hooks_check_their_arguments(lib):
    for bad in (dict(wait_limit_us=-1), dict(hold=-1), dict(hold=4)):
        with pytest.raises(api.MoEError) as e:
            api.product_test_hooks(**bad)
        assert e.value.code == BAD
    with pytest.raises(KeyError):
        api.product_test_hooks(hold="everything")
    api.product_test_hooks(5, "sum")
    api.product_test_hooks()
