"""Builds libqknorm.so (the QK-Norm C ABI) and libstreamceil.so (the
benchmark's streaming copy and read kernels) in-tree with hipcc for gfx950,
and their timing-only twins libqknorm_clocks.so and libstreamceil_clocks.so
(the same sources with QKNORM_BLOCK_CLOCKS: every row or copy block records
its start and end clocks; loaded only by ``bench.py --timeline``), and
_qknorm_torch.so, the Python module that marshals torch tensors for the
operators around headwise QK-Norm.

    python -m layerwise_qk_norm_qknorm_amd.build_lib

Every build recompiles all sources. The libraries are written next to this
file, where the binding (``libqknorm.so``) and bench.py (the others) load
them from.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqknorm.so")
CEIL_LIB = os.path.join(PKG, "libstreamceil.so")
CLOCKS_LIB = os.path.join(PKG, "libqknorm_clocks.so")
CEIL_CLOCKS_LIB = os.path.join(PKG, "libstreamceil_clocks.so")

SOURCES = ["qknorm_api.cpp", "qknorm_ops_api.cpp", "qknorm_kernels.hip", "qknorm_rope.hip",
           "qknorm_rope_paired.hip", "qknorm_attend.hip", "qknorm_attend_wide.hip", "qknorm_gather.hip"]
CEIL_SOURCES = ["stream_ceiling.hip"]
TORCH_LIB = os.path.join(PKG, "_qknorm_torch.so")
TORCH_SOURCE = os.path.join(CSRC, "qknorm_torch.cpp")
ARCH = "gfx950"
JOBS = 6       # compilers at a time, 1 to 3 GB each


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libqknorm.so)")


def command(out, sources, defines=(), link=False):
    """hipcc of the sources into an object, or of objects into a library."""
    if link:
        return [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *sources, "-o", out]
    return [
        hipcc(), "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-c",
        "-Wall", "-Wno-unused-function", *[f"-D{d}" for d in defines],
        # Packed fp32 instructions stay off: the compiler would form them
        # from plain float code, and they are not used anywhere here.
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC,
        *[os.path.join(CSRC, s) for s in sources],
        "-o", out,
    ]


def _run(cmd, verbose):
    if verbose:
        print("[build] " + " ".join(cmd), flush=True)
    proc = subprocess.run(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in proc.stderr.splitlines() if noise not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"compiler failed for {os.path.basename(cmd[-1])} ({proc.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def torch_command(out):
    """The marshalling module: host C++ against torch's headers, linked to
    libqknorm.so beside it (torch's own libraries are loaded before it)."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(base, "include"), os.path.join(base, "lib")
    return [
        os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++"), "-O2", "-std=c++17", "-fPIC", "-shared",
        "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE, TORCH_SOURCE, "-o", out,
        "-L", PKG, "-l:libqknorm.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
    ]


def build(verbose=True):
    """Compiles every source of the four libraries into an object of its own, links
    them, then the marshalling module; returns the path of libqknorm.so."""
    libs = [(LIB, SOURCES, ()), (CLOCKS_LIB, SOURCES, ("QKNORM_BLOCK_CLOCKS",)), (CEIL_LIB, CEIL_SOURCES, ()),
            (CEIL_CLOCKS_LIB, CEIL_SOURCES, ("QKNORM_BLOCK_CLOCKS",))]
    with tempfile.TemporaryDirectory() as tmp, concurrent.futures.ThreadPoolExecutor(JOBS) as pool:
        objects = {lib: [os.path.join(tmp, f"{os.path.basename(lib)}.{s}.o") for s in sources]
                   for lib, sources, _ in libs}
        jobs = [pool.submit(_run, command(o, [s], defines), verbose)
                for lib, sources, defines in libs for s, o in zip(sources, objects[lib])]
        for job in jobs:
            job.result()
        for lib, _, _ in libs:
            _run(command(lib + ".tmp", objects[lib], link=True), verbose)
            os.replace(lib + ".tmp", lib)
    _run(torch_command(TORCH_LIB + ".tmp"), verbose)
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build())
