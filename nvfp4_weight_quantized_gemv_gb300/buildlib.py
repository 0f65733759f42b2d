"""Build the in-tree C-ABI library ``libnvfp4_gemv.so`` for sm_103a.

Usage: ``python -m nvfp4_weight_quantized_gemv_gb300.buildlib`` (or ``build()``).
Translation units compile in parallel with nvcc, then link into one shared
library next to this file.  Static cudart, one -gencode (compute_103a/sm_103a).
``build(debug_bounds=True)`` makes ``libnvfp4_gemv_debug.so`` from the same
sources with -DNVFP4_DEBUG_BOUNDS: the kernels' computed workspace indices
are checked on the device (a failed check sets a bit of the device error
word and skips the access).

``build_binding()`` makes ``_attn_binding.so``, the attention operators' Python
binding, with g++ against Python's and PyTorch's headers; where there is no
PyTorch it makes nothing.  The library needs neither.  The binding fits one
interpreter and one PyTorch: a stamp beside the objects names them, and a binding
with another stamp is built anew, and not loaded.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnvfp4_gemv.so")
OBJ_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libnvfp4_gemv_debug.so")
SOURCES = ["gemv_stream.cu", "gemv_tc.cu", "gemv_fp4.cu", "gemv_generic.cu", "abi.cu", "quantize_host.cpp", "gemv_noalloc.cu",
           "quantize_gpu.cu", "moe_gemv.cu", "moe_mma.cu",
           "selftest.cu", "abi_attn.cu", "attn_heads.cu", "attn_decode.cu", "attn_prompt.cu", "attn_shared.cu", "attn_chunks.cu", "abi_batch.cu", "kv_tables.cu",
           "verify.cu"]
HEADERS = ["ptx.cuh", "tcgen05.cuh", "internal.h", "abi_internal.h", "attn_internal.h", "attn_units.h", "attn.cuh", "batch_internal.h", "scan.cuh"]
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_attn_binding.so")
BINDING_STAMP = os.path.join(OBJ, "binding.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _flags(src: str, debug_bounds: bool = False):
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-ffp-contract=off",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC] + (["-DNVFP4_DEBUG_BOUNDS"] if debug_bounds else [])
    if src.endswith(".cu"):
        return ARCH + common + ["-Xptxas", "-v"]
    return common


def _newest_input() -> float:
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "nvfp4_gemv.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, debug_bounds: bool = False) -> str:
    lib, objdir = (LIB_DEBUG, OBJ_DEBUG) if debug_bounds else (LIB, OBJ)
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _newest_input():
        return lib
    nvcc = nvcc_path()
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc] + _flags(src, debug_bounds) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def binding_fits():
    """What a binding is made for: the interpreter's ABI, where PyTorch is and which one.  None without PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch_dir = os.path.dirname(spec.origin)
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([sysconfig.get_config_var("EXT_SUFFIX"), torch_dir, f.read()])


def binding_made_for():
    """What the present binding was made for; None if there is none."""
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return None
    with open(BINDING_STAMP) as f:
        return f.read()


def build_binding(force: bool = False):
    """Returns the binding's path, None without PyTorch."""
    fits = binding_fits()
    if fits is None:
        return None
    header = os.path.join(ROOT, "include", "nvfp4_gemv.h")
    newest = max(os.path.getmtime(f) for f in (BINDING_SOURCE, header, os.path.abspath(__file__)))
    if not force and binding_made_for() == fits and os.path.getmtime(BINDING) >= newest:
        return BINDING
    torch_dir = fits.splitlines()[1]
    include = [os.path.dirname(header), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"),
               os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include")]
    libs = os.path.join(torch_dir, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared"] + [x for i in include for x in ("-isystem", i)]
           + [BINDING_SOURCE, "-o", tmp, "-L" + libs, "-Wl,-rpath," + libs]
           + ["-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.makedirs(OBJ, exist_ok=True)
    if os.path.exists(BINDING_STAMP):
        os.remove(BINDING_STAMP)
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(fits)
    os.replace(tmp, BINDING_STAMP)
    return BINDING


def build_all(force: bool = False) -> None:
    """The release and the debug-bounds library and the Python binding, compiled side by side."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=3) as ex:
        for f in [ex.submit(build, force, False, False), ex.submit(build, force, False, True),
                  ex.submit(build_binding, force)]:
            f.result()


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug_bounds="--debug-bounds" in sys.argv))
    print(build_binding(force="--force" in sys.argv) or "no Python binding of the attention operators: no PyTorch here")
