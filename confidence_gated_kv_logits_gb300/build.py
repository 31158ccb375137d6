"""Build the CONF-KV CUDA library in-tree (nvcc, sm_103a, no cmake).

Each .cu file under csrc/ is compiled to an object in parallel, then linked
into ``libconfkv.so`` next to this file; csrc/paged_py.cpp, which reads tensor
arguments for the paged operators, becomes the Python module ``_paged_ops.so``
(g++ with torch's own headers, linked to both).  The library needs neither Python's
headers nor torch: it is linked first, and without torch the module is left out
(the binding then says so when it is used).  Host code is compiled without
floating-point contraction so the per-layer budget table is computed with
plain IEEE double operations.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconfkv.so")
OPS = os.path.join(HERE, "_paged_ops.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off",
                   "-I", os.path.join(HERE, "..", "include")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(x) > t for x in deps)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _torch():
    """torch's folder, None without torch."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _ops_against(torch):
    """What the module is built against: it is built anew when this changes."""
    with open(os.path.join(torch, "version.py")) as f:
        return "\n".join([sys.version, sysconfig.get_paths()["include"], torch, f.read()])


def _ops_object(src, obj, torch):
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=1",
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
          "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(cuda, "include"), "-c", src, "-o", obj], f"g++ on {src}")
    with open(obj + ".against", "w") as f:
        f.write(_ops_against(torch))


def _ops_stale(src, obj, hdrs, torch):
    if _stale(obj, [src] + hdrs) or not os.path.exists(obj + ".against"):
        return True
    with open(obj + ".against") as f:
        return f.read() != _ops_against(torch)


def _ops_link(obj, torch):
    lib = os.path.join(torch, "lib")
    tmp = OPS + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libconfkv.so", "-L", lib, "-ltorch_python",
          "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"],
         "linking _paged_ops.so")
    os.replace(tmp, OPS)


def build(force=False, verbose=False):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(HERE, "..", "include", "*.h")))
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(OBJ, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append((s, o))

    def compile_one(so):
        s, o = so
        cmd = [nvcc()] + _flags() + ["-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {s}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return o

    ops_src = os.path.join(CSRC, "paged_py.cpp")
    ops_obj = os.path.join(OBJ, "paged_py.o")
    torch = _torch()
    ops = torch and (force or _ops_stale(ops_src, ops_obj, hdrs, torch))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        extra = ex.submit(_ops_object, ops_src, ops_obj, torch) if ops else None
        list(ex.map(compile_one, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if extra:
        extra.result()
    if torch and (force or _stale(OPS, [ops_obj, LIB])):
        _ops_link(ops_obj, torch)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
