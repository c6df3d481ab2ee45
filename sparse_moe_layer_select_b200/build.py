"""Build the in-tree shared libraries (nvcc for sm_100a, the host compiler for the binding).

  libmoe_b200.so    the MoE layer (C ABI of include/moe.h and include/moe_rows.h)
  libmoe_gen.so     the seeded input generator (test and benchmark inputs only)
  _rows_binding.so  argument marshalling of the row and 8-bit integer calls (CPython module;
                    left out where torch, Python's headers or g++ are missing: programs of the
                    C ABI need none of them)

Usage: python -m sparse_moe_layer_select_b200.build   (or build() from Python)
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr"]

MOE_SOURCES = ["moe_api.cu", "moe_gemm.cu", "moe_gemm_pair.cu", "moe_fused.cu", "router_cc.cu",
               "index.cu", "elementwise.cu", "permute_static.cu", "sorted_rows.cu", "int8_rows.cu",
               "int8_gemm.cu", "int8_gemm_pair.cu", "int8_gemv.cu", "rows_api.cu"]
GEN_SOURCES = ["gen.cu"]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("nvcc not found")


def _newer(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_lib(name, sources, extra=(), force=False, verbose=False):
    out = os.path.join(PKG, name)
    deps = [os.path.join(CSRC, s) for s in sources]
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps += [os.path.join(ROOT, "include", h) for h in ("moe.h", "moe_rows.h")]
    if not force and not _newer(out, deps):
        return out
    # (--threads 0: the sources side by side, one per host core)
    cmd = [_nvcc(), *ARCH, *FLAGS, "--threads", "0", "-shared", "-o", out + ".tmp",
           *[os.path.join(CSRC, s) for s in sources], *extra]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def _binding_lacks():
    """What the binding needs and is not here, or None."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None if shutil.which("g++") else "g++"


def _build_binding(force=False, verbose=False):
    """The CPython module over the C ABI (it reads torch tensors, so it needs torch's headers)."""
    lacks = _binding_lacks()
    if lacks:
        print(f"_rows_binding.so not built: no {lacks} (moe.py's row and 8-bit integer calls "
              "need it)", file=sys.stderr)
        return None
    out = os.path.join(PKG, "_rows_binding.so")
    src = os.path.join(CSRC, "rows_binding.cpp")
    if not force and not _newer(out, [src, *(os.path.join(ROOT, "include", h)
                                           for h in ("moe.h", "moe_rows.h"))]):
        return out
    import torch
    from torch.utils import cpp_extension
    inc = [f"-I{d}" for d in cpp_extension.include_paths()]
    inc += ["-I" + sysconfig.get_paths()["include"],
            "-I" + os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    abi = int(torch.compiled_with_cxx11_abi())
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           *inc, src, "-o", out + ".tmp", f"-L{PKG}", "-l:libmoe_b200.so", f"-L{lib}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def build(force=False, verbose=False):
    """Compile the libraries (skips up-to-date ones); returns the paths of the first two."""
    moe = _build_lib("libmoe_b200.so", MOE_SOURCES, force=force, verbose=verbose)
    gen = _build_lib("libmoe_gen.so", GEN_SOURCES, force=force, verbose=verbose)
    _build_binding(force=force, verbose=verbose)
    return moe, gen


if __name__ == "__main__":
    for p in build(force="--force" in sys.argv, verbose=True):
        print(p)
