"""Build libretnet.so (the C-ABI library and its sm_100a kernels) and its torch binding in-tree.

The library needs nvcc alone; the binding is built where torch and its headers are, for that torch and
that Python (binding_key), and again where these have changed.
"""
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libretnet.so")
BINDING = os.path.join(PKG, "_torch_binding.so")  # torch tensors in, calls into libretnet.so out
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")
BINDING_KEY = os.path.join(BUILD_DIR, "torch_binding.key")  # what the binding there is was built for

NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr", "-diag-suppress", "177"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                               + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _torch():
    """The torch package with what a build against it needs, or None."""
    try:
        import torch
    except ImportError:
        return None
    header = os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "utils", "pybind.h")
    return torch if os.path.exists(header) else None


def binding_key() -> str:
    """The C++ and Python interfaces that a binding built now is for."""
    import sysconfig

    import torch
    return f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}"


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))]) or not os.path.exists(BINDING_KEY):
        return False
    with open(BINDING_KEY) as f:
        return f.read() == binding_key()


def _binding_command(out):
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_torch_binding",
            f'-DRETNET_BINDING_KEY="{binding_key()}"',
            *[f"-I{d}" for d in includes], BINDING_SRC, "-o", out, f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python", f"-L{PKG}", "-l:libretnet.so", "-Wl,-rpath,$ORIGIN"]


def _build_binding():
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    subprocess.run(_binding_command(tmp), check=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BINDING_KEY, "w") as f:
        f.write(binding_key())
    os.replace(tmp, BINDING)


def _bring_binding_up(force: bool):
    if _torch() is None:
        print("torch or its headers are missing: libretnet.so is built, its torch binding is not", file=sys.stderr)
    elif force or not binding_up_to_date():
        _build_binding()


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every csrc/*.cu for sm_100a and link libretnet.so, then, where torch is, the torch binding; return
    the library's path."""
    if not force and up_to_date():
        _bring_binding_up(force)
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    procs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd))
        procs.append((subprocess.Popen(cmd), src))
        objs.append(obj)
    failed = [src for p, src in procs if p.wait() != 0]
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = f"{LIB}.{os.getpid()}.tmp"
    link = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp, "-cudart", "static"]
    subprocess.run(link, check=True)
    os.replace(tmp, LIB)
    _bring_binding_up(force)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
