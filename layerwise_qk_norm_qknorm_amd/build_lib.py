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

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqknorm.so")
CEIL_LIB = os.path.join(PKG, "libstreamceil.so")
CLOCKS_LIB = os.path.join(PKG, "libqknorm_clocks.so")
CEIL_CLOCKS_LIB = os.path.join(PKG, "libstreamceil_clocks.so")

SOURCES = ["qknorm_api.cpp", "qknorm_ops_api.cpp", "qknorm_kernels.hip", "qknorm_rope.hip",
           "qknorm_rope_paired.hip", "qknorm_attend.hip"]
CEIL_SOURCES = ["stream_ceiling.hip"]
TORCH_LIB = os.path.join(PKG, "_qknorm_torch.so")
TORCH_SOURCE = os.path.join(CSRC, "qknorm_torch.cpp")
ARCH = "gfx950"


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libqknorm.so)")


def command(out, sources=SOURCES, defines=()):
    return [
        hipcc(), "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-shared",
        "-Wall", "-Wno-unused-function", *[f"-D{d}" for d in defines],
        # Packed fp32 instructions stay off: the compiler would form them
        # from plain float code, and they are not used anywhere here.
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC,
        *[os.path.join(CSRC, s) for s in sources],
        "-o", out,
    ]


def _start(lib, sources, defines, verbose):
    tmp = lib + ".tmp"
    cmd = command(tmp, sources, defines)
    if verbose:
        print("[build] " + " ".join(cmd), flush=True)
    return lib, tmp, subprocess.Popen(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _finish(job, verbose):
    lib, tmp, proc = job
    _, stderr = proc.communicate()
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in stderr.splitlines() if noise not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"compiler failed for {os.path.basename(lib)} ({proc.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)
    os.replace(tmp, lib)
    return lib


def _build_one(lib, sources, verbose, defines=()):
    return _finish(_start(lib, sources, defines, verbose), verbose)


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
    """Compiles the four libraries (two hipcc processes at a time), then the
    marshalling module; returns the path of libqknorm.so."""
    jobs = [(CEIL_LIB, CEIL_SOURCES, ()), (CEIL_CLOCKS_LIB, CEIL_SOURCES, ("QKNORM_BLOCK_CLOCKS",)),
            (CLOCKS_LIB, SOURCES, ("QKNORM_BLOCK_CLOCKS",)), (LIB, SOURCES, ())]
    for a, b in (jobs[:2], jobs[2:]):
        running = [_start(lib, src, defs, verbose) for lib, src, defs in (a, b)]
        for job in running:
            _finish(job, verbose)
    tmp = TORCH_LIB + ".tmp"
    cmd = torch_command(tmp)
    if verbose:
        print("[build] " + " ".join(cmd), flush=True)
    _finish((TORCH_LIB, tmp, subprocess.Popen(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                              text=True)), verbose)
    return LIB


if __name__ == "__main__":
    print(build())
