"""Builds libra.so (the C-ABI library) in-tree for sm_103a with nvcc, and
the Python module _serving (the torch binding of the serving calls, a file for
each torch and Python ABI) with g++.

Each translation unit compiles in parallel into _build/, then one link
step writes context_varlen_ring_gb300/libra.so, and one the module, which
calls into it.  No CMake.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libra.so")
SOURCES = ["ra_api.cpp", "ra_plan.cpp", "ra_stats.cpp", "ra_misc.cu", "ra_simt.cu", "ra_tc_fwd.cu", "ra_tc_bwd.cu",
           "ra_tc_dq.cu", "ra_noalloc.cu", "ra_tile_build.cu", "ra_rope.cu", "ra_paged.cu", "ra_paged_mma.cu",
           "ra_paged_tc.cu", "ra_serve.cpp", "ra_delta.cu", "ra_delta_tc.cu", "ra_delta_tc_grads.cu", "ra_delta_bwd.cu", "ra_delta.cpp",
           "ra_weights.cu", "ra_weights_tc.cu", "ra_evict.cu", "ra_keep.cpp"]
MODULE_SRC = os.path.join(CSRC, "py_serving.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-I" + os.path.join(HERE, "..", "include")]


def environment() -> str:
    """The installed torch and Python ABI, which the binding is compiled for."""
    import torch
    return f"{torch.__version__}-{sysconfig.get_config_var('SOABI')}"


def module_path() -> str:
    """The binding of this environment: a file for each, so that none loads (or takes for new) another's."""
    return os.path.join(HERE, f"_serving-{environment()}.so")


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _module_job():
    """(object file, compile command, link command, libraries) of the Python module, for the installed torch; each
    command wants its output's name next."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD, f"py_serving-{environment()}.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    cmd += [x for i in inc for x in ("-isystem", i)] + ["-c", MODULE_SRC, "-o"]
    lib = os.path.join(root, "lib")
    link = ["-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + HERE, "-l:libra.so",
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return obj, cmd, ["g++", "-shared", obj, "-o"], link


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(" ".join(cmd) + "\n" + r.stdout + r.stderr)


def _compile_module(force, headers):
    """Compiles the binding where it is stale; its object file, and the link command with its libraries."""
    obj, cmd, link, libs = _module_job()
    if force or _stale(obj, [MODULE_SRC, __file__] + headers):
        tmp = obj + f".tmp{os.getpid()}"
        _run(cmd + [tmp])
        os.replace(tmp, obj)
    return obj, link, libs


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Builds the library, which needs nvcc alone, and the torch binding.  A binding that cannot be built is reported
    and left out: the serving calls of Python then raise, all else works."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(HERE, "..", "include", "ra.h"))
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    objs = []
    jobs = []
    for s in srcs:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, __file__] + headers):
            cmd = [nvcc()] + ARCH + COMMON + list(extra) + ["-c", src, "-o", obj]
            if s.endswith(".cpp"):
                cmd = [nvcc(), "-x", "c++"] + COMMON + list(extra) + ["-c", src, "-o", obj]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        module = ex.submit(_compile_module, force, headers)
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                failed.append(cmd[-3])
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    out = None
    try:
        out = module_path()
        obj, link, libs = module.result()
        if force or _stale(out, [obj, LIB]):
            tmp = out + f".tmp{os.getpid()}"
            _run(link + [tmp] + libs)
            os.replace(tmp, out)
    except Exception as e:  # (torch missing, its headers, g++, or a torch that the binding does not fit)
        if out and os.path.exists(out):
            os.remove(out)  # it is older than the library
        sys.stderr.write(f"{LIB} is built; the torch binding of the serving calls is not: {e}\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
