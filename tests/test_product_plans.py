"""Which kernel a product takes (moe_get_product_plan, on the host): the tested
shapes reach every kernel, tile and split that the choice can take."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

from mixture_experts_routed_03_b200 import api, build
from tests.product_shapes import SHAPES, plan_key

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return api.lib()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_shape_takes_the_kernel_it_is_listed_for(shape):
    assert plan_key(shape[0], *shape[5:]) == shape[:5]


def test_every_choice_has_its_shape():
    """Sizes spread over the whole range (logarithms): no choice that is not listed."""
    rng = random.Random(3)

    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    listed, seen = {s[:5] for s in SHAPES}, set()
    assert len(listed) == len(SHAPES)
    for _ in range(100000):
        M = spread(1, 40000)
        sizes = ("int8", M, spread(1, 20000), spread(1, 131071))
        seen.add(plan_key(*sizes))
        sizes = ("router", M, spread(1, 1024), 256 * spread(1, 128))
        seen.add(plan_key(*sizes))
    assert seen <= listed, sorted(seen - listed)


def test_plan_of_a_tile_fits_its_kernel():
    for kind, kernel, _, _, _, M, N, K in SHAPES:
        p = api.product_plan(kind == "int8", M, K, N)
        assert p.rows >= 1 and p.cols >= 1 and p.splits in (1, 2, 4, 8)
        assert (p.estimate_us > 0) == (kernel != "few")
        if kernel == "tiles":
            assert p.rows % 16 == 0 and p.rows <= 128


def test_plan_refuses_what_the_calls_refuse():
    for args, code in (((0, 0, 256, 8), api.MOE_ERR_INVALID_ARG), ((0, 4, 300, 8), api.MOE_ERR_INVALID_ARG),
                       ((0, 4, 256, 1025), api.MOE_ERR_UNSUPPORTED), ((1, 4, 131072, 8), api.MOE_ERR_UNSUPPORTED),
                       ((1, 4, 0, 8), api.MOE_ERR_INVALID_ARG), ((1, 4, 8, 0), api.MOE_ERR_INVALID_ARG),
                       ((1, (1 << 30) + 1, 8, 8), api.MOE_ERR_UNSUPPORTED)):
        with pytest.raises(api.MoEError) as e:
            api.product_plan(*args)
        assert e.value.code == code, args
    assert api.lib().moe_get_product_plan(1, 4, 64, 8, None) == api.MOE_ERR_INVALID_ARG
    assert api.lib().moe_get_product_plan(2, 4, 64, 8, ctypes.byref(api.ProductPlan())) == api.MOE_ERR_INVALID_ARG


def test_struct_layout_matches_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {printf("%zu", '
                   'sizeof(moe_product_plan_t));' +
                   "".join(f'printf(" %zu", offsetof(moe_product_plan_t, {f}));' for f, _ in api.ProductPlan._fields_) +
                   "return 0;}\n")
    exe = tmp_path / "l"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert [int(v) for v in out.split()] == [ctypes.sizeof(api.ProductPlan)] + [
        getattr(api.ProductPlan, f).offset for f, _ in api.ProductPlan._fields_]
