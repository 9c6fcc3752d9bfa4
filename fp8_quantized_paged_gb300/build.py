"""Build libkvq.so in-tree with nvcc for sm_103a (GB300).

Each CUDA source compiles to an object in parallel (the decode kernels once
per cache format and head size), then nvcc links the
shared library (static CUDA runtime, no libcuda link: the tensor-map encoder
is looked up through the runtime's driver entry-point query).

The native Python binding (the 4-bit cache, the operators around a serving step) is
a library of its own, built with g++ against Python's and torch's headers.  libkvq.so needs nvcc alone: where the binding does
not build, build() says so on stderr and links the library all the same.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkvq.so")
SOURCES = ["kvq_host.cu", "kvq_write.cu", "kvq_decode.cu", "kvq_decode_tc.cu", "kvq_decode_blk.cu",
           "kvq_static.cu", "kvq_calib.cu", "kvq_prefill.cu", "kvq_decode_variant.cu",
           "kvq_fp4_write.cu", "kvq_fp4_decode.cu", "kvq_fp4_prefill.cu", "kvq_rope.cu", "kvq_pages.cu",
           "kvq_tree.cu"]
HEADERS = ["kvq_common.cuh", "kvq_host.h", "kvq_decode.cuh", "kvq_tc.cuh", "kvq_decode_tc.cuh",
           "kvq_decode_blk.cuh", "kvq_prefill_tc.cuh", "kvq_fp4.cuh", "kvq_fp4_host.h", "kvq_fp4_decode.cuh",
           "kvq_fp4_prefill.cuh", "kvq_quant.cuh", "kvq_tree.cuh"]
# (object, source, defines): one object per translation unit, the decode
# variants once per (format, head size); kvq_fmt 0 = BF16, 1 = E4M3, 2 = E5M2
UNITS = [(os.path.splitext(s)[0], s, []) for s in SOURCES if s != "kvq_decode_variant.cu"] + [
    (f"kvq_decode_f{fmt}_d{dh}", "kvq_decode_variant.cu",
     [f"-DKVQ_VARIANT_FMT={fmt}", f"-DKVQ_VARIANT_DH={dh}"])
    for fmt in (1, 2, 0) for dh in (128, 64)]
# the Python binding of the 4-bit cache and of the operators around a step: host code against torch's headers
BINDING = ["fp4_binding.cpp", "step_binding.cpp"]
BINDING_HEADERS = ["binding.h"]
BINDING_LIB = os.path.join(BUILD, "_kvq_fp4.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs(sources):
    inc = os.path.join(os.path.dirname(HERE), "include")
    return ([os.path.join(CSRC, s) for s in sources] +
            [os.path.join(inc, h) for h in ("kvq.h", "kvq_fp4.h", "kvq_step.h")] + [os.path.abspath(__file__)])


def _newer(lib: str, sources) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs(sources))


# The tests' timeout build: the same sources with the test hooks compiled in
# (a decode whose producer withholds one page on request) and bounded waits
# cut to 2^16 polls, in a directory of its own.  Never loaded by the package.
TEST_LIB = os.path.join(BUILD, "test", "libkvq_test.so")
TEST_DEFINES = ["-DKVQ_TEST_HOOKS", "-DKVQ_MAX_POLLS=65536u"]


def up_to_date(lib: str = LIB) -> bool:
    return _newer(lib, SOURCES + HEADERS)


def _torch_root() -> str:
    """torch's folder, without importing it."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found")
    return list(spec.submodule_search_locations)[0]


def _binding_stamp() -> str:
    """What the binding is compiled against: this Python and torch's version file."""
    with open(os.path.join(_torch_root(), "version.py")) as f:
        return sys.version + "\n" + f.read()


def binding_up_to_date() -> bool:
    if not _newer(BINDING_LIB, BINDING + BINDING_HEADERS) or not os.path.exists(BINDING_LIB + ".stamp"):
        return False
    with open(BINDING_LIB + ".stamp") as f:
        return f.read() == _binding_stamp()


def build_binding(verbose: bool = False) -> str:
    import sysconfig
    torch = _torch_root()
    os.makedirs(BUILD, exist_ok=True)
    for old in (BINDING_LIB, BINDING_LIB + ".stamp"):  # a failure leaves no binding of other headers behind
        if os.path.exists(old):
            os.remove(old)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BINDING_LIB + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           "-Wno-attributes", *[os.path.join(CSRC, s) for s in BINDING], "-o", tmp,
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(torch, "include"),
           "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-I/usr/local/cuda/include",
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {' '.join(BINDING)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)
    with open(BINDING_LIB + ".stamp", "w") as f:
        f.write(_binding_stamp())
    return BINDING_LIB


def _try_binding(force: bool, verbose: bool) -> None:
    try:
        if force or not binding_up_to_date():
            build_binding(verbose)
    except (RuntimeError, OSError) as e:
        print(f"the 4-bit cache's Python binding is not built: {e}", file=sys.stderr)


def build_test_lib(force: bool = False, verbose: bool = False) -> str:
    return build(force=force, verbose=verbose, extra=TEST_DEFINES, lib=TEST_LIB)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          lib: str = LIB) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        if lib == LIB:  # the tests' library needs no binding
            ex.submit(_try_binding, force, verbose)
        return lib if not force and up_to_date(lib) else _build_lib(verbose, extra, lib)


def _build_lib(verbose: bool, extra: list[str] | None, lib: str) -> str:
    out_dir = os.path.dirname(lib)
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    extra = list(extra or [])

    def compile_one(unit):
        name, src, defines = unit
        obj = os.path.join(out_dir, name + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *defines, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(len(UNITS), max(2, os.cpu_count() or 2))) as ex:
        objs = list(ex.map(compile_one, UNITS))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    v = "-v" in sys.argv
    ex = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force=True, verbose=v, extra=ex))
