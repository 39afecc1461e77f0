"""Build libqmm.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ compiles in its own nvcc process (in
parallel), then one link step produces quantized_matmul_gb300/libqmm.so.  The
compiled half of the Python binding (csrc/binding.cpp, host code on torch's
headers) compiles with the host compiler beside them and links against that
library: quantized_matmul_gb300/_qmm_torch.so.  The library needs neither torch
nor Python's headers: where they are missing it is built alone, with a message.
Objects go to quantized_matmul_gb300/_build/.  Nothing is installed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqmm.so")
BINDING = os.path.join(HERE, "_qmm_torch.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["qmm_api.cu", "quant.cu", "gemv.cu", "gemv_q8.cu", "gemv_stream.cu", "gemm.cu",
           "gemm_small.cu", "bitnet_gemm.cu", "probe.cu", "bitnet_small.cu",
           "norm.cu", "kv_append.cu", "attend_f16.cu", "attend_q8.cu", "logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I" + INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")


def _newer(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in sources)


def _header() -> str:
    return os.path.join(INCLUDE, "qmm.h")


def library_up_to_date() -> bool:
    return _newer(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] + [_header()])


def binding_up_to_date() -> bool:
    """Newer than its sources, and made for this torch and Python, whose C++ interfaces it goes by."""
    if not _newer(BINDING, [os.path.join(CSRC, "binding.cpp"), _header()]):
        return False
    try:
        with open(_stamp_file()) as f:
            return f.read() == _stamp()
    except (OSError, HeadersMissing):
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


class HeadersMissing(RuntimeError):
    """What the binding alone needs is not there."""


def _torch_dirs() -> tuple[str, str]:
    """torch's include and library folders (found without importing it)."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise HeadersMissing("torch is not installed")
    root = os.path.dirname(spec.origin)
    return os.path.join(root, "include"), os.path.join(root, "lib")


def _stamp_file() -> str:
    return os.path.join(BUILD, "binding.stamp")


def _stamp() -> str:
    root = os.path.dirname(_torch_dirs()[0])
    try:
        with open(os.path.join(root, "version.py")) as f:
            version = f.read()
    except OSError:
        version = "unknown\n"
    return f"python {sys.version}\ntorch {root}\n{version}"


def _compile_binding() -> str:
    import sysconfig
    torch_include = _torch_dirs()[0]
    python_include = sysconfig.get_path("include")
    for file in (os.path.join(python_include, "Python.h"), os.path.join(torch_include, "ATen", "ATen.h")):
        if not os.path.exists(file):
            raise HeadersMissing(f"{file} is missing")
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + torch_include,
           "-isystem", python_include, "-isystem", cuda, "-I" + INCLUDE,
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    lib = _torch_dirs()[1]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libqmm.so", "-L" + lib, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(_stamp_file(), "w") as f:
        f.write(_stamp())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    library = force or ptxas_info or not library_up_to_date()
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(compile_one, SOURCES)) if library else []
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath," + cuda_lib_dir(),
               "-o", tmp, *[o for o, _ in results]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    try:
        _link_binding(binding.result())
    except HeadersMissing as e:
        print(f"{os.path.basename(BINDING)} is not built: {e}.  {os.path.basename(LIB)} does not need it; the Python "
              "functions rms_norm_*, kv_append_*, paged_attention_* and log_probs do.", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
