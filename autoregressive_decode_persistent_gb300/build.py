"""Build libadp.so (the engine's C ABI) in-tree with nvcc for sm_103a.

Thirteen translation units compiled in parallel, then linked as a shared library with the
static CUDA runtime. -fmad=false keeps every multiply-add that the arithmetic contract does
not fuse explicitly as a separate multiply and add; no fast-math flags.

A second library, libadp_test.so, links the same objects with the host engine compiled once more
under -DADP_TEST_HOOKS: it also exports the test-only hooks (withholding a phase's outputs,
shortening the in-kernel waits, moving the epoch counter).  The tests load it; the release
library, which the benchmark and applications load, does not carry those hooks.

Beside them binding.cpp becomes an extension module for the installed PyTorch and Python, whose headers the libraries do not
need: where it cannot be built, build() warns and the libraries are there all the same; calls of ops.py that need it say
that it is missing.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libadp.so")
TEST_LIB = os.path.join(HERE, "libadp_test.so")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))  # (no other Python takes it)
SOURCES = ["decode.cu", "decode_batch.cu", "prefill.cu", "repack.cu", "engine.cu", "noalloc.cu", "probe.cu",
           "paged_rows.cu", "paged_append.cu",
           "paged_attention.cu", "paged_window.cu", "paged_chunk.cu", "packed_attention.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off",
         "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the engine")


def _extra_flags() -> list[str]:
    """Extra nvcc flags from ADP_NVCC_FLAGS (e.g. -DADP_CYCLE_STAMPS for the timeline's cycle
    breakdowns); a change of them forces a rebuild."""
    return os.environ.get("ADP_NVCC_FLAGS", "").split()


FLAGS_STAMP = os.path.join(HERE, "_build", "flags.txt")
BINDING_STAMP = os.path.join(HERE, "_build", "binding.txt")
BINDING_SOURCE = "binding.cpp"


def _older(products: list[str], sources: list[str]) -> bool:
    """Whether a product is missing, or older than a source."""
    if not all(os.path.exists(p) for p in products):
        return True
    t = min(os.path.getmtime(p) for p in products)
    deps = [os.path.join(CSRC, f) for f in sources]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "adp.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _stale() -> bool:
    try:
        if open(FLAGS_STAMP).read() != " ".join(_extra_flags()):
            return True
    except OSError:
        return True
    return _older([LIB, TEST_LIB], [f for f in os.listdir(CSRC) if f != BINDING_SOURCE])


def _binding_for() -> str:
    """What an extension module is made for: PyTorch's version and C++ ABI, and Python's."""
    import torch
    return f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, python {sysconfig.get_config_var('SOABI')}"


def _stale_binding() -> bool:
    try:
        with open(BINDING_STAMP) as fh:
            if fh.read() != _binding_for():
                return True
    except (ImportError, OSError):
        return True  # (where PyTorch is missing, building the module says so)
    return _older([BINDING], [BINDING_SOURCE])


def _build_binding():
    """The extension module with the tensor checks of ops.py's calls, against the installed PyTorch's headers."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    include = [os.path.join(root, "include"), sysconfig.get_paths()["include"], cuda]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DADP_TORCH_VERSION="{torch.__version__}"',
           *(f"-isystem{i}" for i in include), os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as fh:
        fh.write(_binding_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is out of date; the path of libadp.so."""
    with cf.ThreadPoolExecutor(1) as ex:
        binding = ex.submit(_build_binding) if force or _stale_binding() else None
        if force or _stale():
            _build_libraries(verbose)
        error = binding.exception() if binding else None
    if error:
        if os.path.exists(BINDING):
            os.remove(BINDING)  # made of other sources, or for another PyTorch
        warnings.warn(f"{os.path.basename(BINDING)} could not be built ({type(error).__name__}: {error}): the calls of ops.py that need it "
                      "will fail", RuntimeWarning, stacklevel=2)
    return LIB


def _build_libraries(verbose: bool):
    cc = nvcc()
    outdir = os.path.join(HERE, "_build")
    os.makedirs(outdir, exist_ok=True)

    def compile_one(job):
        src, extra, obj_name = job
        obj = os.path.join(outdir, obj_name)
        cmd = [cc, *ARCH, *FLAGS, *_extra_flags(), *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    jobs = [(src, [], src.replace(".cu", ".o")) for src in SOURCES]
    jobs.append(("engine.cu", ["-DADP_TEST_HOOKS"], "engine_hooks.o"))
    with cf.ThreadPoolExecutor(len(jobs)) as ex:
        objs = list(ex.map(compile_one, jobs))
    release = objs[:len(SOURCES)]
    test = [o if not o.endswith(os.sep + "engine.o") else objs[-1] for o in release]
    for lib, members in ((LIB, release), (TEST_LIB, test)):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *members]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, lib)
    with open(FLAGS_STAMP, "w") as fh:
        fh.write(" ".join(_extra_flags()))


if __name__ == "__main__":
    print(build(force=True, verbose=True))
