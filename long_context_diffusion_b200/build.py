"""Builds the C-ABI shared library (libdlsparse.so) in-tree for sm_100a, and
the CPython binding of its token-by-token calls (_calls.so).

    python long_context_diffusion_b200/build.py        (or __graft_entry__.build())

Compiles every csrc/*.cu with nvcc into long_context_diffusion_b200/lib/.
Object files go to _build/ at the repository root; a file is recompiled when
it or any header under csrc/ or include/ is newer than its object.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(LIBDIR, "libdlsparse.so")
CALLS = os.path.join(LIBDIR, "_calls.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _torch_include() -> str:
    """torch's header folder (for its dlpack.h), without importing torch."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found")
    return os.path.join(spec.submodule_search_locations[0], "include")


def _calls_stamp() -> str:
    """What a built extension belongs to besides its sources."""
    include = _torch_include()
    version = os.path.join(os.path.dirname(include), "version.py")
    return "\n".join([sys.version, str(sysconfig.get_config_var("SOABI")), include,
                      open(version).read() if os.path.exists(version) else ""])


def build_calls() -> str | None:
    """The CPython extension of csrc/bind_calls.cpp, built again when a source,
    Python or torch changed.  None where torch's headers have no exchange table:
    the library serves its other calls without the extension."""
    src, hdr = os.path.join(CSRC, "bind_calls.cpp"), os.path.join(ROOT, "include", "dl.h")
    stamp, want = os.path.join(BUILD, "calls.stamp"), _calls_stamp()
    if os.path.exists(CALLS) and os.path.getmtime(CALLS) >= max(os.path.getmtime(src), os.path.getmtime(hdr)) \
            and os.path.exists(stamp) and open(stamp).read() == want:
        return CALLS
    dlpack = os.path.join(_torch_include(), "ATen", "dlpack.h")
    if not os.path.exists(dlpack) or "DLPackExchangeAPI" not in open(dlpack).read():
        print(f"{os.path.basename(CALLS)} not built: {dlpack} has no DLPackExchangeAPI; the token-by-token calls are "
              "not available", file=sys.stderr)
        if os.path.exists(CALLS):
            os.remove(CALLS)
        return None
    os.makedirs(BUILD, exist_ok=True)
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I",
           os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"], "-I",
           _torch_include(), src, "-o", CALLS + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(CALLS + ".tmp", CALLS)
    with open(stamp, "w") as f:
        f.write(want)
    return CALLS


def build(verbose: bool = False, extra: list | None = None) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_t = _newest_header()
    extra = list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_t) \
                and not extra:
            return obj, ""
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", src,
               "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, srcs))
    objs = [o for o, _ in results]
    if verbose:
        for (_, log), src in zip(results, srcs):
            if log.strip():
                print(f"--- {os.path.basename(src)}\n{log}")
    newest_obj = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest_obj:
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    build_calls()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
