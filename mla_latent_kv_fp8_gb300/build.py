"""Build the CUDA library in-tree for sm_103a with nvcc (no cmake).

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked into
``libmla_decode.so`` next to this file; ``csrc/binding.cpp`` becomes the Python
extension ``_packed.so`` beside it (g++, against the installed torch).  The library needs nvcc alone: where the
extension cannot be built, a warning says so, the decode and the C ABI are there all the same, and the packed operators'
Python functions raise.  The CUDA runtime is linked statically; the driver API is reached through the runtime's
entry-point query.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmla_decode.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_packed.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla_decode.so")
    return cand


def _flags(verbose_ptxas: bool):
    # hidden visibility: only the MLA_API entry points of include/*.h are exported
    f = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr", *ARCH]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _run(cmd):
    try:
        return subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:  # no such compiler
        return subprocess.CompletedProcess(cmd, 127, "", f"{e}\n")


def _binding_jobs(force: bool):
    """The command that compiles the Python extension's object, if it is stale."""
    import sysconfig

    import torch
    obj = os.path.join(BUILD, "binding.o")
    stamp = os.path.join(BUILD, "packed.torch")  # the object is for one torch
    built_for = open(stamp).read() if os.path.exists(stamp) else ""
    header = os.path.join(os.path.dirname(HERE), "include", "mla_decode.h")
    if not (force or built_for != torch.__version__ or _stale(obj, [BINDING_SRC, header, __file__])):
        return [], obj
    with open(stamp, "w") as f:
        f.write("")
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return [["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
             f"-I{sysconfig.get_paths()['include']}", f"-I{root}/include", f"-I{cuda}/include",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", BINDING_SRC, "-o", obj]], obj


def _link_binding(obj: str) -> None:
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    r = _run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-lmla_decode", "-Wl,-rpath,$ORIGIN", f"-L{root}",
              "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking _packed.so failed")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "packed.torch"), "w") as f:
        f.write(torch.__version__)


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) libmla_decode.so, whose path is returned, and the Python extension (or warn)."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "mla_decode.h"))
    vptx = verbose or bool(os.environ.get("MLA_PTXAS_VERBOSE"))
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *headers, __file__]):
            jobs.append([nvcc, *_flags(vptx), "-c", src, "-o", obj])
    kernels = list(jobs)
    try:
        binding, binding_obj = _binding_jobs(force)
    except Exception as e:  # no torch, or one without headers
        binding, binding_obj = [], None
        problem = str(e)
    jobs += binding
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            results = list(ex.map(_run, jobs))
        for cmd, r in zip(jobs, results):
            if vptx or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0 and cmd in binding:
                binding_obj, problem = None, f"{cmd[0]} failed for {BINDING_SRC}"
            elif r.returncode != 0:
                raise RuntimeError(f"{cmd[0]} failed for {cmd[-3]}")
    if force or kernels or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static"],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("linking libmla_decode.so failed")
        os.replace(tmp, LIB)
    if binding_obj and (binding or _stale(BINDING, [binding_obj])):
        try:
            _link_binding(binding_obj)
        except (RuntimeError, OSError) as e:
            binding_obj, problem = None, str(e)
    if binding_obj is None:
        if os.path.exists(BINDING):  # of another source or torch
            os.remove(BINDING)
        warnings.warn(f"the Python extension of the packed operators was not built: {problem}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
