"""Build libdspark.so (CUDA, sm_103a) in-tree with nvcc, and with the host compiler
the Python module behind the paged-cache calls (_paged_binding.so)."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libdspark.so")
SOURCES = ["dspark_verify.cu", "dspark_schedule.cu", "dspark_draft.cu", "dspark_paged.cu",
           "dspark_attention.cu"]
BINDING_SOURCE = os.path.join(CSRC, "paged_binding.cpp")
BINDING_PATH = os.path.join(PKG, "_paged_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "paged_binding.stamp")
HEADERS = sorted(f for f in os.listdir(CSRC) if f.endswith(".cuh"))

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _binding_abi() -> str:
    """What the module's machine code is tied to: this Python, and this torch's C++ classes."""
    import torch
    return "\n".join([sysconfig.get_config_var("EXT_SUFFIX") or "", sys.version, torch.__version__,
                      str(torch.version.git_version), str(int(torch.compiled_with_cxx11_abi()))])


def binding_fits() -> bool:
    """Whether the module that is there was compiled for the Python and torch that run."""
    try:
        with open(BINDING_STAMP) as f:
            return os.path.exists(BINDING_PATH) and f.read() == _binding_abi()
    except OSError:
        return False


def _build_binding() -> None:
    """The module's only libraries are torch's own, loaded already wherever it is imported."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING_PATH + ".tmp"
    abi = int(torch.compiled_with_cxx11_abi())
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-isystem", os.path.join(root, "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           BINDING_SOURCE, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SOURCE}:\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_abi())


def _stale() -> bool:
    if not os.path.exists(LIB_PATH) or not binding_fits():
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps += [os.path.join(ROOT, "include", h) for h in ("dspark.h", "dspark_testing.h", "dspark_paged.h")]
    deps += [os.path.abspath(__file__), BINDING_SOURCE]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, extra_flags=()) -> str:
    """Compile every CUDA source for sm_103a and the Python module (in parallel) and link
    libdspark.so."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB_PATH + ".tmp"
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp,
                        *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True))
