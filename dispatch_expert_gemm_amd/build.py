"""Build libmoe.so (the HIP kernels and their C ABI) for gfx950, in-tree.

    python -m dispatch_expert_gemm_amd.build

compiles every csrc/*.hip with hipcc into lib/libmoe.so, and csrc/torch_nodes.cpp
(autograd nodes that call it; this part needs g++, torch's and Python's headers) into
lib/moe_torch.so.  It always recompiles.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe.so")
TORCH_NODES = os.path.join(LIBDIR, "moe_torch.so")
ARCH = "gfx950"

# -packed-fp32-ops: keep the compiler from forming packed fp32 adds/muls/fmas.
COMMON = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", INCLUDE, "-I", CSRC]
# Per-file extras: the gather-reduce kernels keep every product and sum
# separately rounded so their results match a plain left-to-right fp32 sum.
EXTRA = {"combine.hip": ["-ffp-contract=off"]}


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if c and os.path.exists(c):
            return c
    return "hipcc"


def rocm_include() -> str:
    """The headers beside the chosen hipcc."""
    found = shutil.which(hipcc())
    for path in (found, os.path.realpath(found)) if found else (hipcc(),):
        include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(path))), "include")
        if os.path.exists(os.path.join(include, "hip", "hip_runtime.h")):
            return include
    return "/opt/rocm/include"


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".hip"))


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature: harmless
    out = "\n".join(l for l in p.stdout.splitlines()
                    if "packed-fp32-ops" not in l and "warning: feature flag" not in l
                    and l.strip() != "1 warning generated.")
    return p.returncode, out


def nodes_command():
    """The compiler call of the autograd nodes' object file (host code only)."""
    from torch.utils import cpp_extension
    includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], rocm_include()]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            "-DTORCH_API_INCLUDE_EXTENSION_H", "-DTORCH_EXTENSION_NAME=moe_torch", "-I", INCLUDE, "-I", CSRC,
            *[a for i in includes for a in ("-isystem", i)],
            "-c", os.path.join(CSRC, "torch_nodes.cpp"), "-o", os.path.join(LIBDIR, "obj", "torch_nodes.o")]


def _must(what, cmd, verbose=False):
    rc, out = _run(cmd)
    if verbose and out.strip():
        print(out)
    if rc != 0:
        raise RuntimeError(f"{what}:\n{' '.join(cmd)}\n{out}")


def compile_nodes(verbose=False):
    _must("the compiler failed on torch_nodes.cpp", nodes_command(), verbose)


def link_nodes():
    from torch.utils import cpp_extension
    libs = cpp_extension.library_paths()
    tmp = TORCH_NODES + ".tmp"
    _must("link failed", ["g++", "-shared", os.path.join(LIBDIR, "obj", "torch_nodes.o"), "-L" + LIBDIR, "-l:libmoe.so",
                          "-Wl,-rpath,$ORIGIN", *["-L" + p for p in libs], "-lc10", "-lc10_hip", "-ltorch_cpu",
                          "-ltorch", "-ltorch_python", "-o", tmp])
    os.replace(tmp, TORCH_NODES)


def build(verbose: bool = False) -> str:
    os.makedirs(os.path.join(LIBDIR, "obj"), exist_ok=True)
    cc = hipcc()
    jobs = []
    for src in sources():
        obj = os.path.join(LIBDIR, "obj", src.replace(".hip", ".o"))
        cmd = [cc, *COMMON, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((src, obj, cmd))
    with ThreadPoolExecutor(max_workers=min(8, len(jobs) + 1)) as ex:
        kernels = [ex.submit(_must, f"hipcc failed on {src}", cmd, verbose) for src, _, cmd in jobs]
        nodes = ex.submit(compile_nodes, verbose)
        for k in kernels:
            k.result()
        # libmoe.so needs nothing of the nodes: linked before their failure is raised
        tmp = LIB + ".tmp"
        _must("link failed", [cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *[o for _, o, _ in jobs], "-o", tmp])
        os.replace(tmp, LIB)
    try:
        nodes.result()
        link_nodes()
    except Exception:
        if os.path.exists(TORCH_NODES):
            os.remove(TORCH_NODES)  # (an older one may not go with this libmoe.so)
        raise
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
