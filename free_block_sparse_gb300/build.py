"""Build libsparge.so in-tree: nvcc for sm_103a, one object per source file, compiled in
parallel, then one shared-library link; and _binding.so, the Python binding of the serving calls,
against the installed torch's headers and libraries (left out where there is no torch: the C library needs none).
No CMake; runs the same on x86_64 and aarch64 hosts."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsparge.so")
BINDING = os.path.join(PKG, "_binding.so")

CUDA_SOURCES = ["api.cu", "pool_sim.cu", "score_gemm.cu", "score_select.cu", "bsattn.cu", "decode.cu", "permute.cu", "noalloc.cu", "q8prep.cu",
                "norm_rope.cu", "cache4.cu", "cache4_attn.cu", "cache4_bounds.cu", "prefix_attn.cu", "window_decode.cu", "window_attn.cu", "window_v.cu"]
CXX_SOURCES = ["hilbert.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s" % (" ".join(cmd), r.stdout))
    return r.stdout


def _stale(obj, deps):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _binding_job(obj):
    """The compile command of the binding; torch's version file is a dependency (another torch, another build)."""
    t = _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    src = os.path.join(CSRC, "binding.cpp")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", src, "-o", obj]
    for d in inc:
        cmd += ["-isystem", d]
    return cmd, [src, os.path.join(ROOT, "include", "sparge.h"), os.path.join(t, "version.py")]


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
          "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libsparge.so", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
    os.replace(tmp, BINDING)


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "sparge.h"))
    jobs = []
    objs = []
    for src in CUDA_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc] + ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-c", s, "-o", o]
            if ptxas_verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    for src in CXX_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", s, "-o", o])
    binding_obj = os.path.join(BUILD, "binding.cpp.o")
    binding, binding_stale = _torch_dir() is not None, False
    if binding:
        binding_cmd, binding_deps = _binding_job(binding_obj)
        binding_stale = force or _stale(binding_obj, binding_deps)
    lib_stale = force or bool(jobs) or not os.path.exists(LIB)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        compiled = ex.submit(_run, binding_cmd) if binding_stale else None
        for out in ex.map(_run, jobs):
            if verbose and out.strip():
                print(out)
    if lib_stale:
        tmp = LIB + ".tmp"
        _run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if compiled is not None:
        compiled.result()   # a binding that does not compile is an error, after the library is there
    if binding and (binding_stale or lib_stale or not os.path.exists(BINDING)):
        _link_binding(binding_obj)
    elif not binding and verbose:
        print("torch not found: the Python binding of the serving calls is left out")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
