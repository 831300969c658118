"""Build libqcodec.so in-tree with nvcc for sm_103a, and the torch binding of the
8-bit layer's calls (``_qcbind``) next to it with g++ (left out where torch is not
installed: only that layer needs it, and it can call the library through ctypes).

Each CUDA translation unit is compiled to an object file in parallel, then the
objects are linked into a shared library next to this file.  The CUDA runtime
is linked statically, so the library depends only on the driver at run time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libqcodec.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BIND_PATH = os.path.join(PKG, "_qcbind.so")
BIND_SOURCE = "qc_bind.cpp"
BIND_STAMP = os.path.join(PKG, "_qcbind.stamp")  # the torch and Python that _qcbind was compiled against
SOURCES = ["qc_api.cu", "qc_encode.cu", "qc_encode_tma.cu", "qc_encode_clip.cu",
           "qc_encode_clip_bf16.cu", "qc_encode_bf16.cu", "qc_encode_bf16_fast.cu", "qc_decode.cu", "qc_decode_tma.cu",
           "qc_reencode.cu", "qc_reencode_other.cu", "qc_topk.cu", "qc_fp8.cu",
           "qc_encode_log.cu", "qc_reencode_log.cu", "qc_selftest.cu", "qc_encode_direct_log.cu",
           "qc_api_layer.cu", "qc_int8_rows.cu", "qc_int8_product.cu", "qc_int8_few.cu", "qc_int8_wide.cu", "qc_int8_ragged.cu"]
HEADERS = ["qc_device.cuh", "qc_internal.h", "qc_encode_math.cuh", "qc_encode_tma.cuh",
           "qc_encode_direct.cuh",
           "qc_reencode.cuh", "qc_pipeline.cuh", "qc_decode_math.cuh", "qc_exact_norm.cuh",
           "qc_api_util.h", "qc_int8_rows.cuh", "qc_tc.cuh", "qc_tc_host.h", "qc_chain.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# -fmad=false: no multiply-add contraction; every fused op is an explicit
# __fmaf_rn.  Division and square root stay IEEE (no fast math).
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-ffp-contract=off"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libqcodec")


def _newer(path, sources) -> bool:
    """path exists and is no older than its sources and this file."""
    files = [*sources, os.path.join(ROOT, "include", "qcodec.h"), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def bind_stamp():
    """What an extension depends on besides its sources, without importing torch: where torch
    lies, its version file, and the interpreter's ABI.  None where torch is not installed."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    with open(os.path.join(root, "version.py")) as f:
        return "\n".join((root, str(sysconfig.get_config_var("SOABI")), f.read()))


def bind_fits() -> bool:
    """_qcbind was compiled against the torch and the Python that are here now."""
    try:
        with open(BIND_STAMP) as f:
            return os.path.exists(BIND_PATH) and f.read() == bind_stamp()
    except OSError:
        return False


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, [os.path.join(CSRC, s) for s in SOURCES + HEADERS])


def bind_up_to_date() -> bool:
    return bind_stamp() is None or (bind_fits() and _newer(BIND_PATH, [os.path.join(CSRC, BIND_SOURCE)]))


def up_to_date() -> bool:
    return library_up_to_date() and bind_up_to_date()


def bind_flags():
    """Compiler and linker flags of an extension against the installed torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               cuda, sysconfig.get_paths()["include"]]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ([f"-D_GLIBCXX_USE_CXX11_ABI={abi}"] + [f"-I{p}" for p in include],
            [f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def _link(cmd, path):
    """Run the linker into a temporary file and put it in place in one step."""
    tmp = path + f".tmp{os.getpid()}"
    r = subprocess.run([*cmd[:2], "-o", tmp, *cmd[2:]], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libqcodec.so and the binding; returns the library's path."""
    lib, bind = force or not library_up_to_date(), bind_stamp() is not None and (force or not bind_up_to_date())
    if not lib and not bind:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    def compile_bind():
        obj = os.path.join(BUILD_DIR, "qc_bind.o")
        flags, libs = bind_flags()
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *flags, "-c", os.path.join(CSRC, BIND_SOURCE), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {BIND_SOURCE}:\n{r.stdout}\n{r.stderr}")
        return obj, libs

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        bound = ex.submit(compile_bind) if bind else None
        results = list(ex.map(compile_one, SOURCES)) if lib else []
        if verbose or ptxas_info:
            for _, log in results:
                if log:
                    print(log)
        # the library is in place whatever becomes of the binding
        if lib:
            _link([cc, "-shared", *ARCH, *[o for o, _ in results], "-cudart", "static", "-Xlinker", f"-soname={LIB_NAME}"],
                  LIB_PATH)
        if bind:
            stamp = bind_stamp()
            obj, libs = bound.result()
            _link(["g++", "-shared", obj, LIB_PATH, "-Wl,-rpath,$ORIGIN", *libs], BIND_PATH)
            with open(BIND_STAMP, "w") as f:
                f.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True,
                        ptxas_info="--ptxas-info" in sys.argv))
