"""Build libpkv.so in-tree (paged_kv_decode_attention_gb300/_build/) with nvcc
for sm_103a only.  Translation units compile in parallel, then link into one
shared library with the CUDA runtime linked statically.  Beside it, with g++
against the installed torch's headers, the Python entry points of the calls
that serve single tokens (_pkv_binding.<torch and Python>.so,
csrc/py_binding.cpp)."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import platform
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
# one build folder per host architecture (the box that runs the GPU may differ)
BUILD = os.path.join(HERE, "_build", platform.machine())
LIB = os.path.join(BUILD, "libpkv.so")
BINDING_SRC = os.path.join(CSRC, "py_binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", f"-I{INCLUDE}", f"-I{CSRC}",
                     "--expt-relaxed-constexpr"] + os.environ.get("PKV_NVCC_FLAGS", "").split()


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    import torch

    return os.path.dirname(os.path.abspath(torch.__file__))


def _binding_tag() -> str:
    """What the binding's machine code depends on besides its sources: torch's C++ classes and Python's."""
    import torch

    commit = (getattr(torch.version, "git_version", None) or "")[:8]
    return re.sub(r"[^\w.+-]", "_", f"{torch.__version__}-{commit}-{sysconfig.get_config_var('SOABI')}")


def binding_path() -> str:
    return os.path.join(BUILD, f"_pkv_binding.{_binding_tag()}.so")


def _binding_compile(obj: str):
    torch_dir = _torch_dir()
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj, f"-I{INCLUDE}",
            "-I" + sysconfig.get_paths()["include"], "-I" + inc,
            "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), f"-I{os.path.join(cuda, 'include')}"]


def _binding_link(obj: str, out: str):
    return ["g++", "-shared", "-o", out, obj, "-L" + BUILD, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _run_all(jobs, verbose: bool) -> None:
    def run(cmd):
        return cmd, subprocess.run(cmd, capture_output=True, text=True)

    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or r.returncode != 0:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode != 0:
                    raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}")


def _link(command, out: str) -> None:
    """Run command(output) into a temporary file beside `out`, then put it in its place."""
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run(command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"link of {os.path.basename(out)} failed")
    os.replace(tmp, out)


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False, binding: bool = True) -> str:
    """Build what is stale: libpkv.so, and the binding unless it is left to build_binding()."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = headers()
    objs = []
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [src] + hdrs):
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            jobs.append(cmd)
    cuda_jobs = len(jobs)
    if binding:
        jobs += _binding_jobs(force)
    _run_all(jobs, verbose or ptxas_info)
    if force or cuda_jobs or _stale(LIB, objs):
        _link(lambda out: [nvcc] + ARCH + ["-shared", "-o", out] + objs, LIB)
    if binding:
        _link_binding(force)
    return LIB


def _binding_obj() -> str:
    return os.path.join(BUILD, f"py_binding.{_binding_tag()}.o")


def _binding_jobs(force: bool = False):
    obj = _binding_obj()
    return [_binding_compile(obj)] if force or _stale(obj, [BINDING_SRC] + headers()) else []


def _link_binding(force: bool = False) -> None:
    if force or _stale(binding_path(), [_binding_obj()]):
        _link(lambda out: _binding_link(_binding_obj(), out), binding_path())


def build_binding() -> str:
    """The binding alone, beside a library that is built."""
    _run_all(_binding_jobs(), False)
    _link_binding()
    return binding_path()


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv, force="-f" in sys.argv))
