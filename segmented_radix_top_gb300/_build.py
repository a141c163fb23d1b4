"""Builds libsegtopk.so from csrc/ with nvcc for sm_103a (in-tree, no cmake).

Each .cu is compiled to an object in parallel, then linked into one shared
library next to this file. A rebuild happens only when a source or header is
newer than the library.

The instrumented variant (libsegtopk_instr.so, variant="instr") is the same
sources compiled with SEGTOPK_STATS and SEGTOPK_TEST_HOOKS: per-CTA counters
(segtopk_read_stats) and the test hooks of the bounded copy wait
(segtopk_set_test_hooks). build_all() compiles both in one pool of
compiler processes.

Beside the library, csrc/rows_binding.cpp becomes _rows_native.*.so (g++,
Python's and PyTorch's headers): the Python binding of the row operators. It
does not link the library; _rows.py hands it the entry points of the loaded
one. The library needs none of that: it is built first, and alone where those
headers are not installed.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libsegtopk.so")
BINDING_SRC = os.path.join(CSRC, "rows_binding.cpp")
VARIANTS = {
    "": (BUILD_DIR, LIB_PATH, []),
    "instr": (os.path.join(HERE, "_build_instr"), os.path.join(HERE, "libsegtopk_instr.so"),
              ["-DSEGTOPK_STATS", "-DSEGTOPK_TEST_HOOKS"]),
}

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# hidden visibility: only the C ABI (SEGTOPK_API in include/segtopk.h) is
# exported, so two builds loaded in one process (the ordinary and the
# instrumented one) share no symbol, not even a function-local static
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-I", INCLUDE,
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def lib_path(variant: str = "") -> str:
    return VARIANTS[variant][1]


def up_to_date(variant: str = "") -> bool:
    path = lib_path(variant)
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(variant: str, src: str, extra_flags, verbose: bool) -> str:
    build_dir, _, variant_flags = VARIANTS[variant]
    obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + variant_flags + list(extra_flags or []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def binding_path() -> str:
    """The binding's file. Its name holds the interpreter's and PyTorch's
    versions: it is compiled against their classes, which differ from one to
    the next, so that after a change of either it is built anew."""
    import torch
    return os.path.join(HERE, "_rows_native.%s.torch-%s.so" % (sysconfig.get_config_var("SOABI"), torch.__version__))


def _binding_includes():
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    return [base, os.path.join(base, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]


def binding_lacks():
    """What the binding cannot be compiled without and this machine does not have."""
    lacks = [] if shutil.which("g++") else ["g++"]
    for header in ("Python.h", os.path.join("torch", "csrc", "autograd", "python_variable.h")):
        if not any(os.path.exists(os.path.join(d, header)) for d in _binding_includes()):
            lacks.append(header)
    return lacks


def binding_up_to_date() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in [BINDING_SRC, os.path.join(INCLUDE, "segtopk.h"),
                                                  os.path.abspath(__file__)])


def _compile_binding(verbose: bool) -> str:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = binding_path()
    tmp = path + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           *("-I" + d for d in _binding_includes()), BINDING_SRC, "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BINDING_SRC, r.stdout, r.stderr))
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, path)
    return path


def _link(variant: str, objs) -> str:
    out_path = VARIANTS[variant][1]
    tmp = out_path + ".tmp.%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + list(objs)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, out_path)
    return out_path


def build_variants(variants, force: bool = False, verbose: bool = False, extra_flags=None):
    """Builds the given variants and the row operators' binding, every
    translation unit of all of them in one pool of compiler processes;
    returns the library paths. The libraries do not wait for the binding: an
    error of its compilation is raised once they are linked, and where this
    machine cannot compile it that is said on stderr (and again by the first
    call of a row operator)."""
    todo = [v for v in variants if force or not up_to_date(v)]
    for v in todo:
        os.makedirs(VARIANTS[v][0], exist_ok=True)
    srcs = _sources()
    jobs = [(v, s) for v in todo for s in srcs]
    binding = force or not binding_up_to_date()
    lacks = binding_lacks() if binding else []
    if lacks:
        binding = False
        sys.stderr.write("the binding of the row operators is not built: %s not installed\n" % ", ".join(lacks))
    if jobs or binding:
        with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
            bound = ex.submit(_compile_binding, verbose) if binding else None
            objs = list(ex.map(lambda j: _compile(j[0], j[1], extra_flags, verbose), jobs))
        for v in todo:
            _link(v, [o for (vv, _), o in zip(jobs, objs) if vv == v])
        if bound:
            bound.result()
    return [lib_path(v) for v in variants]


def build(force: bool = False, verbose: bool = False, extra_flags=None, variant: str = "") -> str:
    return build_variants([variant], force=force, verbose=verbose, extra_flags=extra_flags)[0]


def build_all(force: bool = False, verbose: bool = False):
    """The library and its instrumented variant."""
    return build_variants(list(VARIANTS), force=force, verbose=verbose)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None,
                variant="instr" if "--instr" in sys.argv else ""))
