"""Build the CUDA library ``libsvdq_b200.so`` in-tree with nvcc (sm_100a), and
the module through which Python calls its MXFP4 part.

Usage: ``python bit_w4a4_diffusion_b200/build.py [-v]`` (or ``build()`` from
``__graft_entry__``); run it by path -- importing the package loads the
library this script produces.  Objects are rebuilt only when a source or header is
newer than the object.  Cross-compiles without a GPU.
"""
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "lib", "libsvdq_b200.so")
# Named for the interpreter it is built for, so that another one does not load it.
BIND = os.path.join(PKG, "_mxfp4" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-fmad=false",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
CXX_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-pthread", "-I", INCLUDE,
             "-I", "/usr/local/cuda/include"]

CU_SOURCES = ["abi.cu", "quantize_act.cu", "quantize_nvfp4.cu", "gemm_nvfp4.cu", "gemm_nvfp4_pair.cu", "gemm_int4.cu", "gemm_int4_pair.cu", "dequant_int4.cu", "awq_gemm.cu", "noalloc.cu",
              "mxfp4_abi.cu", "mxfp4_quant.cu", "mxfp4_gemm_pair.cu",
              "mxfp4_gemm_pair_swiglu.cu", "mxfp4_gemm_narrow.cu"]
CXX_SOURCES = ["pack.cpp", "calib.cpp", "mxfp4_pack.cpp"]
BIND_SOURCE = "mxfp4_bind.cpp"


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"build step failed: {' '.join(cmd[:3])} ...")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)


def build(verbose=False, ptxas_verbose=False):
    """Compile every source for sm_100a and link the shared library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    hdrs = _headers()
    objs = []
    for src in CU_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if _stale(o, [s] + hdrs) or ptxas_verbose:
            extra = ["-Xptxas", "-v"] if ptxas_verbose else []
            _run([NVCC] + NVCC_FLAGS + extra + ["-c", s, "-o", o], verbose or ptxas_verbose)
    for src in CXX_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if _stale(o, [s] + hdrs):
            _run(["g++"] + CXX_FLAGS + ["-c", s, "-o", o], verbose)
    if _stale(LIB, objs):
        _run([NVCC] + ARCH + ["-shared", "-o", LIB] + objs + ["-lpthread"], verbose)
    _build_bind(hdrs, verbose)
    return LIB


def _build_bind(hdrs, verbose):
    """The extension module, against the installed torch and the library.  It
    is rebuilt when its command changes, which names the torch version: an
    installed file's time need not be newer than the module."""
    src = os.path.join(CSRC, BIND_SOURCE)
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    version = runpy.run_path(os.path.join(torch, "version.py"))["__version__"]
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", f'-DBUILT_FOR_TORCH="{version}"',
             "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
             "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
             "-I", "/usr/local/cuda/include"]
    libs = ["-L", os.path.dirname(LIB), "-l:" + os.path.basename(LIB), "-L", os.path.join(torch, "lib"), "-ltorch_python",
            "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN/lib"]
    cmd = ["g++"] + flags + [src, "-o", BIND] + libs
    made_by = os.path.join(BUILD, BIND_SOURCE + ".cmd")
    same = os.path.exists(made_by) and open(made_by).read() == "\n".join(cmd)
    if same and not _stale(BIND, [src] + hdrs):
        return
    _run(cmd, verbose)
    with open(made_by, "w") as f:
        f.write("\n".join(cmd))
    untagged = os.path.join(PKG, "_mxfp4.so")    # what earlier builds made; any interpreter would load it
    if os.path.exists(untagged):
        os.remove(untagged)


if __name__ == "__main__":
    build(verbose=True, ptxas_verbose="-v" in sys.argv)
