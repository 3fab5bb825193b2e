"""In-tree build of the CUDA libraries with nvcc (sm_103a).

``build()`` compiles every translation unit in parallel and links
``kv_cache_token_tip_gb300/libfasa.so`` (the FASA library) and
``workload/libfasa_synth.so`` (the synthetic-input generator used by the tests
and the benchmark); where torch is installed it also builds
``kv_cache_token_tip_gb300/_fasa_torch`` + the Python ABI's suffix (the paged
cache's argument marshalling for torch tensors).  Object files go to
``_build/`` at the repository root.  A library is rebuilt only when one of its
sources is newer than it, the module also when it was built for another torch.
"""

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]

LIBFASA = os.path.join(PKG, "libfasa.so")
LIBSYNTH = os.path.join(ROOT, "workload", "libfasa_synth.so")

FASA_SOURCES = [os.path.join(PKG, "csrc", f) for f in
                ("fasa_api.cu", "fasa_cluster_bf16.cu", "fasa_cluster_f32.cu", "fasa_step_bf16.cu", "fasa_noalloc.cu",
                 "fasa_ca.cu", "fasa_paged.cu", "fasa_paged_attend.cu", "fasa_paged_cache.cu")]
FASA_DEPS = [os.path.join(PKG, "csrc", f) for f in
             ("fasa_cluster.cuh", "fasa_step.cuh", "fasa_ptx.cuh", "fasa_internal.h",
              "fasa_paged.h", "fasa_paged_index.h")] + [
    os.path.join(ROOT, "include", "fasa.h")]
LIBTORCH = os.path.join(PKG, "_fasa_torch" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
TORCH_SOURCES = [os.path.join(PKG, "csrc", "fasa_torch.cpp")]
SYNTH_SOURCES = [os.path.join(ROOT, "workload", "csrc", "synth_gen.cu")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfasa")


def _stale(target, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(x) > t for x in inputs)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def _build_lib(target, sources, deps, extra_flags=(), verbose=False, force=False, ptxas_v=False):
    if not force and not _stale(target, sources + deps):
        return target
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    objs = []
    jobs = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 1))) as ex:
        for src in sources:
            obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
            objs.append(obj)
            cmd = [cc] + NVCC_FLAGS + list(extra_flags) + (["-Xptxas", "-v"] if ptxas_v else []) + [
                "-c", src, "-o", obj]
            jobs.append(ex.submit(_run, cmd, verbose))
        outs = [j.result() for j in jobs]
    if ptxas_v:
        for o in outs:
            print(o.stderr)
    tmp = target + ".tmp"
    _run([cc] + ARCH + ["-shared", "-o", tmp] + objs, verbose)
    os.replace(tmp, target)
    return target


def _build_torch(verbose=False, force=False):
    """The extension module, against the torch that is installed (host code
    alone); None where there is none (the C library does not need it)."""
    import importlib.util
    found = importlib.util.find_spec("torch")
    if found is None or not found.origin:
        return None
    torch = os.path.dirname(found.origin)
    with open(os.path.join(torch, "version.py")) as f:
        about = f.read()
    version = re.search(r"__version__ = ['\"](.*?)['\"]", about).group(1)
    # the torch it was built for: its inline code and layouts are in the module, and a
    # file of another torch may be older than the module
    stamp, built_for = os.path.join(BUILD_DIR, "_fasa_torch.torch"), f"{torch}\n{about}"
    if not force and not _stale(LIBTORCH, TORCH_SOURCES + [os.path.join(ROOT, "include", "fasa.h")]) and \
            os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == built_for:
                return LIBTORCH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = LIBTORCH + ".tmp"
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", f'-DFASA_TORCH_VERSION="{version}"'] + [
        "-I" + d for d in (sysconfig.get_paths()["include"], os.path.join(torch, "include"),
                           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                           os.path.join(cuda, "include"))] + TORCH_SOURCES + [
        "-o", tmp, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], verbose)
    os.replace(tmp, LIBTORCH)
    with open(stamp, "w") as f:
        f.write(built_for)
    return LIBTORCH


def build(verbose=False, force=False, ptxas_v=False):
    """Compile libfasa.so and libfasa_synth.so (in parallel, with the extension module where torch is
    installed); return their paths."""
    with cf.ThreadPoolExecutor(max_workers=3) as ex:
        t = ex.submit(_build_torch, verbose, force)
        a = ex.submit(_build_lib, LIBFASA, FASA_SOURCES, FASA_DEPS, (), verbose, force, ptxas_v)
        b = ex.submit(_build_lib, LIBSYNTH, SYNTH_SOURCES, [], (), verbose, force, False)
        t.result()
        return a.result(), b.result()


if __name__ == "__main__":
    import sys
    print(build(verbose=True, force="--force" in sys.argv, ptxas_v="-v" in sys.argv))
