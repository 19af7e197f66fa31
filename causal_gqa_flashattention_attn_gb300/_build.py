"""Builds libattn.so (the C-ABI library) in-tree with nvcc for sm_103a.

Every .cu file under csrc/ is compiled in parallel to an object under
_build/, then linked into ``libattn.so`` next to this file.  The CUDA runtime
is linked statically and the driver is reached through the runtime's entry
point query, so the library loads on a machine without a GPU driver.

csrc/binding.cpp, the compiled Python binding of the paged cache's entries, is
built beside them with the host compiler, against the installed torch, and
linked into ``_binding.so``; it is built again for another torch or Python than
the ones noted beside it.  libattn.so itself knows nothing of torch.
"""

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
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libattn.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_OBJ = os.path.join(BUILD_DIR, "binding.o")
BINDING_PATH = os.path.join(HERE, "_binding.so")
BINDING_NOTE = os.path.join(BUILD_DIR, "binding.txt")   # what it was built against
API_HEADER = os.path.join(os.path.dirname(HERE), "include", "attn.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-DNDEBUG"] + ARCH


def nvcc():
    exe = shutil.which("nvcc")
    if exe is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found")
    return exe


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(API_HEADER)
    return hs


def _binding_commands():
    """(compile, link) commands of the Python binding; torch is imported only where the binding is stale."""
    import torch
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    includes = [os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"), cuda,
                sysconfig.get_paths()["include"]]
    cxx = os.environ.get("CXX", "g++")
    flags = ["-O2", "-std=c++17", "-fPIC", "-DNDEBUG", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    lib = os.path.join(troot, "lib")
    return ([cxx] + flags + [x for i in includes for x in ("-isystem", i)] + ["-c", BINDING_SRC, "-o", BINDING_OBJ],
            [cxx, "-shared", BINDING_OBJ, "-o", BINDING_PATH + ".tmp", "-L", HERE, "-l:" + LIB_NAME, "-L", lib, "-lc10",
             "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def _binding_against():
    """The torch and the Python that the binding is built against, without importing torch."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # a torch that runs from its source tree
        version = ""
    return f"torch {version} {importlib.util.find_spec('torch').origin}\npython {sys.version}\n"


def _noted():
    try:
        with open(BINDING_NOTE) as f:
            return f.read()
    except FileNotFoundError:
        return None


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose=False, force=False, ptxas_verbose=False):
    """Compile and link; returns the path of libattn.so."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    exe = nvcc()
    hdrs = headers()
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, src[:-3] + ".o")
        srcp = os.path.join(CSRC, src)
        if force or _stale(obj, [srcp] + hdrs):
            cmd = [exe] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", srcp, "-o", obj]
            jobs.append((src, cmd))
    against = _binding_against()
    binding = force or _stale(BINDING_OBJ, [BINDING_SRC, API_HEADER]) or _noted() != against
    if binding or _stale(BINDING_PATH, [BINDING_OBJ]):
        compile_binding, link_binding = _binding_commands()
    if binding:
        jobs.insert(0, (os.path.basename(BINDING_SRC), compile_binding))

    def run(job):
        src, cmd = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, cmd, r

    failed = []
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for src, cmd, r in ex.map(run, jobs):
                if verbose or r.returncode != 0 or ptxas_verbose:
                    sys.stderr.write(f"[{os.path.basename(cmd[0])}] {src}\n{r.stdout}{r.stderr}")
                if r.returncode != 0:
                    failed.append(src)
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    objs = [os.path.join(BUILD_DIR, s[:-3] + ".o") for s in sources()]
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [exe] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB_PATH)
    if binding or _stale(BINDING_PATH, [BINDING_OBJ]):
        r = subprocess.run(link_binding, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link of the binding failed:\n" + r.stdout + r.stderr)
        os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
        with open(BINDING_NOTE, "w") as f:
            f.write(against)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB_PATH)
