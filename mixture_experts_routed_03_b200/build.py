"""Builds ``libmoe_b200.so`` in-tree with nvcc for sm_100a.

    python -m mixture_experts_routed_03_b200.build [--force]

The library is two translation units (``csrc/moe_api.cu``, the routed layer, and
``csrc/block_api.cu``, the operators next to it), each including its kernel
headers and compiled to an object of its own, side by side; the runtime is
linked statically and the driver's tensor-map encoder is looked up at run
time, so the .so needs no libcuda at link time.  ``_binding`` is the Python
extension of ``csrc/binding.c``, under this interpreter's name for it; without
a C compiler or Python's headers it is left out, and the calls that it makes
shorter go through ctypes.
"""

import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libmoe_b200.so")
OBJ = os.path.join(HERE, "_build")   # one object per source
SOURCES = ["moe_api.cu", "block_api.cu"]
# the tensor-core peak probe the benchmark reports its roofline against
PEAK_OUT = os.path.join(HERE, "libmoe_peak.so")
PEAK_SOURCES = ["mma_peak.cu"]
# the Python extension that makes the short calls (csrc/binding.c)
BINDING_OUT = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SOURCE = "binding.c"

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _deps(source):
    """The source and every header it includes, directly or not."""
    seen, todo = set(), [os.path.join(CSRC, source)]
    while todo:
        path = os.path.normpath(todo.pop())
        if path in seen or not os.path.exists(path):
            continue
        seen.add(path)
        with open(path) as f:
            todo += [os.path.join(os.path.dirname(path), n) for n in re.findall(r'^#include "(.+)"', f.read(), re.M)]
    return sorted(seen)


def _newer(out, deps):
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def up_to_date(out=OUT, sources=SOURCES):
    return _newer(out, [d for s in sources for d in _deps(s)])


def _run(cmd):
    res = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    log = " ".join(cmd) + "\n" + res.stdout + res.stderr
    return res.returncode, log


def _compile(out, sources, log_name, force=False):
    """Compile the sources whose objects are missing or old, then link."""
    os.makedirs(OBJ, exist_ok=True)
    objects = {s: os.path.join(OBJ, os.path.splitext(s)[0] + ".o") for s in sources}
    todo = [s for s in sources if force or not _newer(objects[s], _deps(s))]
    cmds = [[_nvcc()] + NVCC_FLAGS + ["-c", "-o", objects[s], os.path.join(CSRC, s)] for s in todo]
    with ThreadPoolExecutor(max(1, len(cmds))) as pool:
        results = list(pool.map(_run, cmds))
    if all(rc == 0 for rc, _ in results):
        results.append(_run([_nvcc()] + NVCC_FLAGS[:2] + ["-shared", "-o", out] + list(objects.values())))
    log = "".join(text for _, text in results)
    with open(os.path.join(HERE, log_name), "w") as f:
        f.write(log)
    if any(rc != 0 for rc, _ in results):
        raise RuntimeError("nvcc failed:\n" + log[-4000:])
    return log


def _build_binding():
    """Compile the Python extension; without it (no C compiler, no Python.h)
    nothing is lost but a microsecond a call, so that is a warning."""
    for old in (BINDING_OUT, os.path.join(HERE, "_binding.so")):   # an older source's, or any interpreter's
        if os.path.exists(old):
            os.remove(old)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        rc, log = 1, "no C compiler"
    else:
        rc, log = _run([cc, "-O2", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"], "-o", BINDING_OUT,
                        os.path.join(CSRC, BINDING_SOURCE)])
    if rc != 0:
        warnings.warn("the _binding extension was not built (short calls go through ctypes): " + log[-2000:])


def build(force=False, verbose=False):
    """Compile the libraries that are missing or older than their sources;
    returns the path of the layer's library."""
    for out, sources, log_name in ((OUT, SOURCES, "build.log"), (PEAK_OUT, PEAK_SOURCES, "build_peak.log")):
        if force or not up_to_date(out, sources):
            log = _compile(out, sources, log_name, force)
            if verbose:
                print(log)
    if force or not up_to_date(BINDING_OUT, [BINDING_SOURCE]):
        _build_binding()
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
