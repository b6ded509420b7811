"""Build libcarve.so in-tree for sm_100a with nvcc, and the torch binding of
the operators around the chunk core.

    python -m chunk_gated_delta_02_b200.build [--force]

Each .cu file under csrc/ (and its folders) is compiled to an object in csrc/_build/ (rebuilt
when it or any header is newer), then linked into
chunk_gated_delta_02_b200/libcarve.so next to the bindings.
csrc/mixer/binding.cpp, host code only, becomes _mixer.so there (g++ against
the headers of the installed torch, linked to that libcarve.so); it is rebuilt
for another torch or Python as well.  libcarve.so needs nvcc alone: where torch,
the C++ compiler or the Python headers are missing, it is built and the binding
is left out with a note on stderr.
"""
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(CSRC, "_build")
LIB = os.path.join(HERE, "libcarve.so")
BINDING_SRC = os.path.join(CSRC, "mixer", "binding.cpp")
BINDING = os.path.join(HERE, "_mixer.so")
BINDING_MADE = os.path.join(OBJ, "_mixer.txt")  # what that was built for
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def _headers():
    return (glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True)
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_lacks():
    """What the binding cannot be built without and this machine has not, or
    None."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if shutil.which(CXX) is None:
        return "the C++ compiler %s" % CXX
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "the Python headers"
    return None


def _binding_for():
    """What a binding is built for, beside its sources."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package
        torch = "unknown"
    return "torch %s, python %s\n" % (torch, sysconfig.get_config_var("SOABI"))


def _binding_stale():
    if _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "carve.h")]):
        return True
    try:
        with open(BINDING_MADE) as f:
            return f.read() != _binding_for()
    except OSError:
        return True


def _binding_command(out):
    import torch
    from torch.utils import cpp_extension
    include = cpp_extension.include_paths() + [
        sysconfig.get_paths()["include"],
        os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ([CXX, "-O2", "-std=c++17", "-fPIC", "-shared",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
            + [a for i in include for a in ("-isystem", i)]
            + [BINDING_SRC, "-o", out, "-L", libs, "-lc10", "-lc10_cuda",
               "-ltorch_cpu", "-ltorch_python", "-L", HERE, "-l:libcarve.so",
               "-Wl,-rpath,$ORIGIN",
               # the C++ runtime that torch has loaded: a static copy next to
               # it crashes (two sets of locale facets)
               "-nostdlib++", "-l:libstdc++.so.6"])


def build(force=False, verbose=False):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "**", "*.cu"), recursive=True))
    hdrs = _headers()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(OBJ, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([NVCC] + ARCH + FLAGS + ["-c", s, "-o", o])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)

    with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        run([NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if force or _binding_stale():
        lacks = _binding_lacks()
        if lacks:
            print("note: %s is not here, so %s is not built (one that is there "
                  "stays as it was); %s is complete"
                  % (lacks, os.path.basename(BINDING), LIB), file=sys.stderr)
            return LIB
        tmp = BINDING + ".tmp.%d" % os.getpid()
        run(_binding_command(tmp))
        os.replace(tmp, BINDING)
        with open(BINDING_MADE, "w") as f:
            f.write(_binding_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
