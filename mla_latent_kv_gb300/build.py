"""Build the CUDA library libmla_latent_kv.so (nvcc, sm_103a only) and the torch binding in-tree.

    python -m mla_latent_kv_gb300.build [--force] [--verbose]

Each .cu under csrc/ is compiled in parallel to an object file, then linked into
mla_latent_kv_gb300/_build/libmla_latent_kv.so (the CUDA runtime is linked statically, so the
library loads on a machine without a GPU; CUDA calls then fail with MLA_ERR_CUDA). binding.cpp, which reads
torch tensors, is compiled beside them by the host compiler into _build/_mla_torch.so and linked to the library;
without torch, which the library does not need, it is left out.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmla_latent_kv.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(BUILD, "_mla_torch.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def has_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def built_for() -> str:
    """What a torch binding built here is for: its object follows the layouts of this torch's headers and of this Python."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_built_for() -> str | None:
    """What the torch binding that is there was built for, None if there is none (or nothing says so)."""
    try:
        with open(BINDING + ".built_for") as f:
            return f.read() if os.path.exists(BINDING) else None
    except OSError:
        return None


def _cuda_home() -> str:
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _binding_cmd(obj):
    import torch
    home = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(_cuda_home(), "include"), "-c", BINDING_SRC, "-o", obj]


def _binding_link(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX", "g++"), "-shared", obj, "-L", BUILD, "-l:" + os.path.basename(LIB),
            "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def up_to_date() -> bool:
    if not _newer(LIB, _deps()):
        return False
    if not has_torch():
        return True
    # a binding of another torch or Python, or brought from elsewhere, is built again
    return _newer(BINDING, _deps() + [BINDING_SRC]) and binding_built_for() == built_for()


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []
    with_torch = has_torch()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = _binding_cmd(obj) if src == BINDING_SRC else [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    def report(results):
        """Prints what the compilers said; raises if one failed."""
        for src, _, r in results:
            if r.returncode != 0 or (verbose and r.stderr):
                sys.stderr.write(f"--- {os.path.basename(src)}\n{r.stdout}{r.stderr}")
        if any(r.returncode != 0 for _, _, r in results):
            raise RuntimeError("a compiler failed; see messages above")

    def link(cmd, out):
        tmp = out + f".{os.getpid()}.tmp"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, out)

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, ([BINDING_SRC] if with_torch else []) + sources()))
    of_library = [x for x in results if x[0] != BINDING_SRC]
    report(of_library)
    link([nvcc, *ARCH, "-shared", "-cudart", "static", *[obj for _, obj, _ in of_library], "-lpthread", "-ldl", "-lrt"], LIB)
    # the binding last: where it cannot be built, the library is there
    if with_torch:
        report(results[:1])
        if os.path.exists(BINDING + ".built_for"):
            os.remove(BINDING + ".built_for")
        link(_binding_link(results[0][1]), BINDING)
        with open(BINDING + ".built_for", "w") as f:
            f.write(built_for())
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
