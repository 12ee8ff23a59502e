"""Build libsrwm.so (the sm_103a CUDA library) in-tree with nvcc, and beside it
_srwm_torch.so, the CPython module that marshals PyTorch tensors for the
linear attention and group norm entry points.

Each translation unit under csrc/ compiles in parallel with
`-gencode arch=compute_103a,code=sm_103a`; the objects link into
self_referential_weight_gb300/libsrwm.so with the CUDA runtime linked
statically, so the library loads next to any PyTorch build.

    python -m self_referential_weight_gb300.build [--force]
"""
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
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsrwm.so")
MODULE = os.path.join(PKG, "_srwm_torch.so")
MODULE_SOURCE = "srwm_torch.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
UNITS = ["srwm_api.cu", "srwm_d16.cu", "srwm_d32.cu", "srwm_d64.cu", "srwm_probe.cu", "srwm_noalloc.cu", "srwm_bwd.cu",
         "srwm_layer.cu", "srwm_ffgemm.cu", "srwm_linattn.cu", "srwm_linattn_tc.cu",
         "srwm_linattn_tc32.cu", "srwm_linattn_scan.cu", "srwm_linattn_api.cu", "srwm_groupnorm.cu",
         "srwm_groupnorm_api.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is needed to build libsrwm.so")


def _sources():
    deps = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))]
    return deps + [os.path.join(INCLUDE, "srwm.h")]


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    return any(os.path.getmtime(s) > t for s in _sources())


def _compile_module(obj: str):
    """srwm_torch.cpp against the installed PyTorch's headers."""
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[a for i in inc for a in ("-isystem", i)],
           "-c", os.path.join(CSRC, MODULE_SOURCE), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compiling {MODULE_SOURCE} failed:\n{res.stdout}\n{res.stderr}")
    return torch_dir


def _link_module(obj: str, torch_dir: str):
    lib = os.path.join(torch_dir, "lib")
    tmp = MODULE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L", PKG, "-l:libsrwm.so", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking _srwm_torch.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MODULE)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libsrwm.so and _srwm_torch.so if missing or older than their sources."""
    if not force and not is_stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                    "-I", CSRC]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_unit(unit):
        obj = os.path.join(BUILD_DIR, unit.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, unit), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {unit}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            sys.stderr.write(res.stderr)
        return obj

    module_obj = os.path.join(BUILD_DIR, "srwm_torch.o")
    with ThreadPoolExecutor(max_workers=len(UNITS) + 1) as ex:
        module = ex.submit(_compile_module, module_obj)
        objs = list(ex.map(compile_unit, UNITS))
        torch_dir = module.result()
    tmp = LIB + f".tmp{os.getpid()}"
    # cuBLASLt (the layer's two feed-forward GEMMs) from the toolkit next to nvcc
    libdir = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-L", libdir, "-lcublasLt",
           "-Xlinker", f"-rpath,{libdir}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking libsrwm.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_module(module_obj, torch_dir)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
