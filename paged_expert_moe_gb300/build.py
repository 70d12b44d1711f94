"""Builds libpagedmoe.so in-tree from the CUDA sources with nvcc (sm_103a only).

Each translation unit is compiled in parallel, then linked into one shared library
with a plain C ABI (include/pagedmoe.h), which needs nvcc alone. Where torch is installed, g++
compiles the Python binding of the decode-step calls (csrc/binding.cpp, against torch's headers)
beside it. Each is rebuilt when a source of its own is newer, the binding also when torch is another.
"""

import concurrent.futures
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedmoe.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fvisibility=hidden"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [p for d in (CSRC, os.path.join(HERE, "..", "include")) for e in ("*.h", "*.cuh")
                         for p in glob.glob(os.path.join(d, e))]


def _stale(lib, deps):
    return not os.path.exists(lib) or any(os.path.getmtime(p) > os.path.getmtime(lib) for p in deps)


def _torch():
    """Where torch is installed, or None; without importing it."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None and spec.submodule_search_locations else None


def _torch_id(torch):
    """What the binding is built against."""
    version = os.path.join(torch, "version.py")
    return torch + "\n" + (open(version).read() if os.path.exists(version) else "")


def _binding_stale():
    torch = _torch()
    if torch is None:
        return False
    stamp = os.path.join(BUILD, "binding.torch")
    if not os.path.exists(stamp) or open(stamp).read() != _torch_id(torch):
        return True
    return _stale(BINDING, [BINDING_SRC] + [p for p in _deps() if p.endswith(".h")])


def needs_build():
    return _stale(LIB, _deps()) or _binding_stale()


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_binding():
    tmp = BINDING + ".tmp"
    torch = _torch()
    lib = os.path.join(torch, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch, "include"), "-I", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           BINDING_SRC, "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "binding.torch"), "w") as f:
        f.write(_torch_id(torch))


def _link(objs):
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force=False, verbose_ptxas=False, quiet=True):
    library, binding = force or _stale(LIB, _deps()), _torch() is not None and (force or _binding_stale())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if library else []
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        made = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
        if made is not None:
            made.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    if library:
        _link([o for o, _ in results])
    if not quiet:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, quiet=False)
