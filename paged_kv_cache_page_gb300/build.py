"""Build libpagedattn.so (and the test-only libpa_selftest.so) in-tree with
nvcc for sm_103a, and the Python module _binding.so (torch tensors to the C
ABI of the serving-step calls) with the host compiler.

Each translation unit is compiled in parallel, then linked into a shared
library with the CUDA runtime linked statically (no libcuda dependency at load
time; the driver is reached at first use).  Run ``python -m
paged_kv_cache_page_gb300.build`` or call :func:`build`.
"""

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_NAME = "libpagedattn.so"
SOURCES = ["api.cu", "append.cu", "decode.cu", "combine.cu", "noalloc.cu", "engine.cu",
           "rotary.cu", "prefill.cu", "step.cu", "rotary_append.cu", "attend_e4m3.cu",
           "chunk_e4m3.cu"]
# Encoding self-test of the tensor-core operand layouts: test infrastructure,
# kept out of the product library.
SELFTEST_LIB = "libpa_selftest.so"
SELFTEST_SOURCES = ["selftest_tcgen05.cu", "selftest_tcgen05_t.cu",
                    "selftest_timeout.cu"]
# Python module of the serving-step calls (host code against torch's headers).
BINDING_LIB = "_binding.so"
BINDING_SOURCE = "binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def lib_path(name=LIB_NAME):
    return os.path.join(OUT_DIR, name)


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")] + list(extra)


def _compile(src, obj, extra, verbose):
    cmd = [nvcc_path(), "-c", os.path.join(CSRC, src), "-o", obj] + _flags(extra)
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _build_binding(lib, verbose):
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    inc = [os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = lib + ".tmp"
    cmd = ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-o", tmp,
            os.path.join(CSRC, BINDING_SOURCE)] + [x for i in inc for x in ("-isystem", i)]
           + ["-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
              "-lc10_cuda"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return r.stdout + r.stderr if verbose else ""


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _link(lib, objs):
    tmp = lib + ".tmp"
    cmd = [nvcc_path(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def build(force=False, verbose=False, extra=()):
    """Compile (if needed) the libraries and the Python module; return the path of
    libpagedattn.so.  The library needs neither Python's headers nor torch's: where the module
    cannot be built that is a warning, and the calls that need it say that it is missing."""
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "pagedattn.h"))
    targets = [(lib_path(LIB_NAME), SOURCES), (lib_path(SELFTEST_LIB), SELFTEST_SOURCES)]
    jobs, objs_of = [], {}
    for lib, sources in targets:
        objs_of[lib] = []
        for src in sources:
            obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
            objs_of[lib].append(obj)
            if force or verbose or _stale(obj, [os.path.join(CSRC, src)] + headers):
                jobs.append((src, obj))
    logs = []
    binding = lib_path(BINDING_LIB)
    bind = force or _stale(binding, [os.path.join(CSRC, BINDING_SOURCE), headers[-1]])
    if jobs or bind:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
            futs = [ex.submit(_compile, s, o, extra, verbose) for s, o in jobs]
            module = ex.submit(_build_binding, binding, verbose) if bind else None
            for f in futs:
                logs.append(f.result())
            if module is not None:
                try:
                    logs.append(module.result())
                except (RuntimeError, OSError, AttributeError) as e:
                    # (one of older sources may not fit the library)
                    if os.path.exists(binding):
                        os.remove(binding)
                    warnings.warn(f"{BINDING_LIB} was not built: {e}", RuntimeWarning, stacklevel=2)
    for lib, objs in objs_of.items():
        if force or _stale(lib, objs):
            _link(lib, objs)
    if verbose:
        print("\n".join(logs))
    return lib_path(LIB_NAME)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
