"""Build the EFLA CUDA library in-tree: ``delta_rule_linear_03_b200/libefla.so``.

Compiles ``csrc/efla_api.cu`` (the mixer), ``csrc/efla_block_api.cu`` (the
operators around it) and ``csrc/efla_scan_*.cu`` (the scan's kernels), side by
side for sm_100a only, and links them with the CUDA runtime, statically, so the
library needs nothing but the driver at run time.  ``csrc/efla_block_binding.cpp``,
the Python binding of the operators around the mixer, becomes
``_efla_block.so``, against PyTorch's headers and the library.  Rebuilds when
any source under ``csrc/`` or ``include/`` is newer than either; the binding
also when the installed PyTorch or Python is not the one that it was built for.

    python delta_rule_linear_03_b200/build.py [--force]

(run it as a file: importing the package needs the library to exist)
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SO = os.path.join(HERE, "libefla.so")
BINDING = os.path.join(HERE, "_efla_block.so")
BUILT_FOR = os.path.join(HERE, "_build", "binding")  # what binding_for() said when the binding was built
SOURCES = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")) +
                 glob.glob(os.path.join(HERE, "csrc", "*.cuh")) +
                 glob.glob(os.path.join(ROOT, "include", "*.h")))
BINDING_SOURCE = os.path.join(HERE, "csrc", "efla_block_binding.cpp")
UNITS = ("efla_api", "efla_block_api", "efla_scan_fwd_f32", "efla_scan_fwd_bf16", "efla_scan_bwd_f32", "efla_scan_bwd_bf16")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def binding_for() -> str:
    """The versions whose interfaces the binding is bound to."""
    import sysconfig

    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def stale_library() -> bool:
    return not os.path.exists(SO) or any(os.path.getmtime(s) > os.path.getmtime(SO) for s in SOURCES)


def stale_binding() -> bool:
    if not os.path.exists(BINDING) or any(os.path.getmtime(s) > os.path.getmtime(BINDING) for s in (SO, BINDING_SOURCE, *SOURCES)):
        return True
    try:
        with open(BUILT_FOR) as f:
            return f.read() != binding_for()
    except OSError:
        return True


def stale() -> bool:
    return stale_library() or stale_binding()


def binding_command(out: str) -> list[str]:
    """g++ on the binding's one source; the library is found beside it at run time."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_efla_block",
            f'-DEFLA_TORCH_VERSION="{torch.__version__}"',
            "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
            BINDING_SOURCE, "-o", out, "-L" + HERE, "-L" + lib, "-l:libefla.so",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale_library():
        build_library(verbose)
        build_binding()
    elif stale_binding():
        build_binding()
    return SO


def build_library(verbose: bool = False) -> None:
    tmp = SO + f".tmp{os.getpid()}"
    objs = [f"{tmp}.{u}.o" for u in UNITS]
    try:
        runs = [subprocess.Popen([nvcc(), *NVCC_FLAGS, "-c", "-o", o, os.path.join(HERE, "csrc", u + ".cu")],
                                 stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                for u, o in zip(UNITS, objs)]
        said = [r.communicate()[0] for r in runs]
        for u, r, text in zip(UNITS, runs, said):
            if r.returncode != 0:
                sys.stderr.write(text)
                raise RuntimeError(f"nvcc failed compiling {u}.cu")
        r = subprocess.run([nvcc(), "-shared", "-cudart", "static", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed linking libefla.so")
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    if verbose:
        sys.stderr.write("".join(said))
    os.replace(tmp, SO)


def build_binding() -> None:
    r = subprocess.run(binding_command(BINDING + f".tmp{os.getpid()}"), capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed building _efla_block.so")
    os.replace(BINDING + f".tmp{os.getpid()}", BINDING)
    os.makedirs(os.path.dirname(BUILT_FOR), exist_ok=True)
    with open(BUILT_FOR, "w") as f:
        f.write(binding_for())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
