"""Build libar.so (HIP kernels for gfx950 + the C ABI) in-tree with hipcc, and
_training.so (the training calls on torch tensors) with the host compiler.

Usage: ``python -m tree_allreduce_algorithms_amd.build_lib`` (or call
``build()``).  hipcc cross-compiles for gfx950 without a GPU present.  Each
source compiles to its own object in parallel (the kernel files instantiate
many dtype x op x unroll variants), then one hipcc call links the library and
one compiler call the module that calls it.  Both are put in place together,
when both are whole.  Without torch, which the collectives do without, the
library is built alone, and says so.
"""

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libar.so")
MODULE = os.path.join(PKG, "_training.so")

SOURCES = ["api.cpp", "plan.cpp", "ring_kernels.hip", "copy_kernels.hip", "tree_kernels.hip",
           "step_kernels.hip", "train/adamw.cpp", "train/adamw_kernels.hip", "train/route.cpp",
           "train/route_kernels.hip", "train/experts.cpp", "train/experts_kernels.hip",
           "train/expert_products.hip", "train/muon.cpp", "train/muon_kernels.hip"]

COMPILE_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # one IEEE operation per hop: no contraction, no flushing of subnormals
    "-ffp-contract=off",
    "-fno-gpu-flush-denormals-to-zero",
    # keep the compiler from emitting packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]
LINK_FLAGS = ["--offload-arch=gfx950", "-shared", "-fPIC"]


def hipcc():
    exe = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError(f"hipcc not found (looked for {exe})")
    return exe


def sources():
    return [os.path.join(CSRC, s) for s in SOURCES]


def has_torch():
    return importlib.util.find_spec("torch") is not None


def host_compiler():
    """CXX, the system's compiler, or the one that comes with hipcc."""
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    return cxx or os.path.join(os.path.dirname(os.path.realpath(hipcc())), "amdclang++")


def module_command(out, libdir):
    """The compiler call that builds the module, from torch's own headers and
    libraries and the libar.so in `libdir`."""
    from torch.utils import cpp_extension
    includes = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    return [host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
            *[a for i in includes for a in ("-isystem", i)],
            os.path.join(CSRC, "train", "torch_calls.cpp"), "-o", out, "-L", libdir, "-lar",
            "-Wl,-rpath,$ORIGIN", *[f"-L{p}" for p in cpp_extension.library_paths()],
            "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _run(what, cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"{what} failed ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")


def build(verbose=False, jobs=None):
    """Compile every source into libar.so and _training.so next to this file;
    returns the library's path.  Where anything fails, both stay as they were."""
    cc = hipcc()
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 1, 8)
    with tempfile.TemporaryDirectory(prefix="ar_build_") as tmpdir:
        objs, procs, pending = [], [], list(sources())
        failures = []
        while pending or procs:
            while pending and len(procs) < jobs:
                src = pending.pop(0)
                obj = os.path.join(tmpdir, os.path.basename(src) + ".o")
                cmd = [cc, *COMPILE_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
                if verbose:
                    print(" ".join(cmd), flush=True)
                procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                    stderr=subprocess.STDOUT, text=True)))
                objs.append(obj)
            src, proc = procs.pop(0)
            out, _ = proc.communicate()
            if proc.returncode != 0:
                failures.append(f"{os.path.basename(src)} ({proc.returncode}):\n{out}")
            elif verbose and out.strip():
                print(out, file=sys.stderr)
        if failures:
            raise RuntimeError("hipcc failed:\n" + "\n".join(failures))
        built = os.path.join(tmpdir, os.path.basename(LIB))
        _run("link", [cc, *LINK_FLAGS, *objs, "-o", built], verbose)
        targets = [(built, LIB)]
        if has_torch():
            module = os.path.join(tmpdir, os.path.basename(MODULE))
            _run("module", module_command(module, tmpdir), verbose)
            targets.append((module, MODULE))
        else:
            print(f"torch is not installed: {os.path.basename(MODULE)} (the training calls) is not built",
                  file=sys.stderr)
        # into this folder first, so that the last step renames within one file system
        for made, target in targets:
            shutil.copy2(made, target + ".tmp")
        for _, target in targets:
            os.replace(target + ".tmp", target)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
