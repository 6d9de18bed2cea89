"""Build the KDA CUDA library (sm_103a) and its compiled Python binding in-tree.

build() compiles every csrc/*.cu with nvcc for sm_103a in parallel and links them into
_build/libkda_gb300.so, a plain shared library exporting the C ABI of include/kda.h; it needs
neither torch nor a host compiler of its own. build_binding() makes csrc/kda_binding.cpp, the
binding of the entry points whose calls are a few microseconds long, with g++ and torch's
headers; it links the library. Its file is named after the Python and the torch that it was
built for, so another one of either builds its own.
"""
import concurrent.futures
import glob
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libkda_gb300.so")
BINDING_SRC = os.path.join(CSRC, "kda_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _newer(target, deps):
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def up_to_date():
    return _newer(LIB, _deps())


def binding_path():
    """The binding's file for the running Python and the installed torch."""
    import torch

    return os.path.join(OUT_DIR, "_kda_binding-%s-torch%s.so" % (sysconfig.get_config_var("SOABI"), torch.__version__))


def binding_up_to_date():
    return _newer(binding_path(), [BINDING_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def build(force=False, verbose=False, extra_flags=()):
    """Compile and link; returns the path of the shared library."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(OUT_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        return _compile([nvcc()] + ARCH + FLAGS + list(extra_flags), *pair)

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(srcs))) as ex:
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for log in logs:
            if log.strip():
                print(log)
    _link([nvcc()] + ARCH + ["-shared"] + objs + ["-lcudart"], LIB)
    return LIB


def build_binding(force=False):
    """Compile and link the binding, the library with it; returns the binding's path."""
    target = binding_path()
    if not force and binding_up_to_date():
        build()
        return target
    os.makedirs(OUT_DIR, exist_ok=True)
    obj, torch_lib = target[:-3] + ".o", os.path.join(_torch_dir(), "lib")
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        made = ex.submit(_compile, ["g++"] + _binding_flags(), BINDING_SRC, obj)
        build()
        made.result()
    _link(["g++", "-shared", obj, "-L" + OUT_DIR, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L" + torch_lib,
           "-Wl,-rpath," + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], target)
    return target


def _torch_dir():
    import torch

    return os.path.dirname(os.path.abspath(torch.__file__))


def _binding_flags():
    import torch

    inc = os.path.join(_torch_dir(), "include")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    dirs = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    # torch's headers as system headers: their warnings are not this file's
    return ["-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden", "-DAT_PER_OPERATOR_HEADERS",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + d for d in dirs] + [
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include")]


def _compile(cmd, src, obj):
    r = subprocess.run(cmd + ["-c", src, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s%s" % (os.path.basename(cmd[0]), src, r.stdout, r.stderr))
    return r.stdout + r.stderr


def _link(cmd, target):
    tmp = target + ".tmp.%d" % os.getpid()
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, target)


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose=True, extra_flags=sys.argv[1:]))
    print(build_binding(force=True))
