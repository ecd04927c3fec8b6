"""The bench's stored DRAM traffic is keyed to the code of the layer's kernels,
and to nothing else."""

import os
import shutil

import pytest

import bench
from mixture_experts_routed_03_b200 import build


@pytest.fixture
def sources(tmp_path, monkeypatch):
    """A copy of the sources that the digest is taken over."""
    csrc = tmp_path / "package" / "csrc"
    shutil.copytree(build.CSRC, csrc)
    shutil.copytree(os.path.join(bench.ROOT, "include"), tmp_path / "include")
    monkeypatch.setattr(build, "CSRC", str(csrc))
    return csrc


def _append(path, text):
    with open(path, "a") as f:
        f.write(text)


def test_digest_is_of_the_layers_sources(sources):
    start = bench.kernel_sources_sha()
    for name in ("norm.cuh", "dense.cuh", "dense_pair.cuh", "block_api.cu", "mma_peak.cu"):
        _append(sources / name, "\nint other;\n")
    (sources / "another_operator.cu").write_text("int other;\n")
    assert bench.kernel_sources_sha() == start
    for name in ("gemm.cuh", "fused.cuh", "common.cuh", "moe_api.cu"):
        _append(sources / name, "\n// a comment\n")
        assert bench.kernel_sources_sha() == start
    for name in ("gemm.cuh", "gemm_swap.cuh", "fused.cuh", "aux_kernels.cuh", "common.cuh", "moe_api.cu",
                 "../../include/moe.h"):
        _append(sources / name, "\nint more;\n")
        now = bench.kernel_sources_sha()
        assert now != start, name
        start = now
