"""Build libdreamer.so (the product), _attention.so (its Python entry points of attention.py),
libdreamer_inputs.so (seeded input generator) and libdreamer_testhooks.so (test infrastructure:
the product's sources with the timeout-test hook and a 20 ms device wait limit) for sm_100a, in-tree."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
# translation units of libdreamer.so
UNITS = ("dreamer.cu", "route_noalloc.cu", "attn_packed.cu", "kv4.cu")
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-shared", "-Xptxas", "-v"] if os.environ.get("DREAMER_PTXAS_VERBOSE") else \
        ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-shared"]


def _newer(target, deps):
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _build_attention(libdreamer, force, verbose):
    """_attention: the Python entry points of attention.py, over libdreamer.so beside it."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    out = os.path.join(HERE, "_attention.so")
    src = os.path.join(CSRC, "attention_py.cpp")
    if not force and _newer(out, [src, libdreamer]):
        return out
    inc = [*ext.include_paths(), sysconfig.get_paths()["include"], os.path.join(CUDA, "include")]
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unused-local-typedefs",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{p}" for p in inc), "-o", out, src, f"-L{HERE}", "-l:libdreamer.so",
           f"-L{tlib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return out


def _sources(exts=(".cu", ".cuh", ".h")):
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(exts)]
    out.append(os.path.join(ROOT, "include", "dreamer.h"))
    return out


def build(force: bool = False, verbose: bool = False) -> list:
    outs = []
    units = [os.path.join(CSRC, u) for u in UNITS]
    lib = os.path.join(HERE, "libdreamer.so")
    deps = [p for p in _sources() if not p.endswith("inputs_gen.cu")]
    if force or not _newer(lib, deps):
        cmd = ["nvcc", *ARCH, *FLAGS, "-t", "0", "-o", lib, *units]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    outs.append(lib)
    outs.append(_build_attention(lib, force, verbose))
    hooks = os.path.join(HERE, "libdreamer_testhooks.so")
    if force or not _newer(hooks, deps):
        cmd = ["nvcc", *ARCH, *FLAGS, "-DDREAMER_TEST_HOOKS",
               "-DDREAMER_WAIT_LIMIT_NS=20000000ull", "-t", "0", "-o", hooks, *units]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    outs.append(hooks)
    gen = os.path.join(HERE, "libdreamer_inputs.so")
    src = os.path.join(CSRC, "inputs_gen.cu")
    if force or not _newer(gen, [src]):
        cmd = ["nvcc", *ARCH, *FLAGS, "-Xcompiler", "-fopenmp", "-o", gen, src, "-lgomp"]
        subprocess.run(cmd, check=True)
    outs.append(gen)
    return outs


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
