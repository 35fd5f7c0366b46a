"""Build libfa_gb300.so in-tree with nvcc for sm_103a (no cmake).

The translation units are compiled in parallel, then linked into
``exact_io_aware_flashattention_gb300/_lib/libfa_gb300.so`` with the CUDA
runtime linked statically.  ``ptxas -v`` output (registers, shared memory,
spills) is kept next to the library as ``ptxas.txt``.

``_lib/fa_torch.so``, the native marshalling of torch tensors, is host code
compiled beside it against the installed torch; the library does not need it,
and where it does not compile the binding marshals in Python.  The module
carries what it was compiled against (``native_key``): with another torch,
Python or ``fa.h`` it is compiled again, and until then not loaded.  What the
compiler said is kept, under the key, as ``fa_torch.txt``.
"""
from __future__ import annotations

import hashlib
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)

TORCH_SOURCE = "fa_torch.cpp"
TORCH_PATH = os.path.join(OUT_DIR, "fa_torch.so")
TORCH_LOG = os.path.join(OUT_DIR, "fa_torch.txt")

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_bwd_dq.cu", "fa_rope.cu", "fa_paged.cu", "fa_evict.cu", "fa_qknorm.cu",
           "fa_append4.cu", "fa_decode4.cu"]
HEADERS = ["sm103a.cuh", "fa_internal.h", "fa_paged.h", "fa_paged4.h", "fa_angle.h", "fa_rotary.cuh", "fa_decode.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS + [TORCH_SOURCE]]
    files += [os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def native_key() -> str:
    """What fa_torch.so depends on besides its source: the installed torch and Python, and fa.h."""
    try:
        import torch
        version = torch.__version__
    except Exception:
        version = "none"
    with open(os.path.join(INCLUDE, "fa.h"), "rb") as f:
        header = hashlib.sha256(f.read()).hexdigest()[:16]
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}, fa.h {header}"


def native_up_to_date() -> bool:
    """Whether fa_torch.txt tells of a module, or of a failure, with today's torch, Python and fa.h."""
    try:
        with open(TORCH_LOG) as f:
            return f.readline().rstrip("\n") == native_key()
    except OSError:
        return False


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr + r.stdout


def _compile_torch() -> None:
    """fa_torch.so, or the reason why not in fa_torch.txt."""
    tmp = TORCH_PATH + ".tmp"
    key, done = native_key(), False
    try:
        import torch
        where = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(nvcc()))
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               f'-DFA_TORCH_KEY="{key}"',
               "-isystem", os.path.join(where, "include"), "-isystem", sysconfig.get_paths()["include"],
               "-isystem", os.path.join(cuda, "include"), "-I", INCLUDE, os.path.join(CSRC, TORCH_SOURCE), "-o", tmp,
               "-L", os.path.join(where, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
               "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, TORCH_PATH)
            done = True
        said = f"{' '.join(cmd)}\nexit {r.returncode}\n{r.stdout}{r.stderr}"
    except Exception as e:       # no torch, no compiler: Python marshals
        said = f"{type(e).__name__}: {e}\n"
    if not done and os.path.exists(TORCH_PATH):
        os.remove(TORCH_PATH)    # of an earlier build: not this library's
    with open(TORCH_LOG, "w") as f:
        f.write(f"{key}\n{said}")


# The forward kernel splits its launch allocation between warpgroups with
# setmaxnreg; the split is only valid for this per-thread register count.
FWD_KERNEL_REGS = 168


def check_registers(ptxas_log: str) -> None:
    """Fail the build if ptxas did not give every forward-kernel instance
    exactly FWD_KERNEL_REGS registers (or spilled in it)."""
    entry = None
    seen = 0
    for line in ptxas_log.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            entry = m.group(1)
            continue
        if entry and "fa_fwd_kernel" in entry:
            m = re.search(r"Used (\d+) registers", line)
            if m:
                seen += 1
                if int(m.group(1)) != FWD_KERNEL_REGS:
                    raise RuntimeError(f"{entry}: ptxas used {m.group(1)} registers, the warpgroup register split "
                                       f"needs exactly {FWD_KERNEL_REGS}")
                entry = None
            m = re.search(r"(\d+) bytes spill stores", line)
            if m and int(m.group(1)) != 0:
                raise RuntimeError(f"{entry}: {m.group(1)} bytes of register spills")
    if seen == 0:
        raise RuntimeError("ptxas reported no forward-kernel instance")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if any source is newer than it, and its marshalling
    also for another torch; return the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and up_to_date():
        if not native_up_to_date():
            _compile_torch()
        return LIB_PATH
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        native = ex.submit(_compile_torch)
        results = list(ex.map(_compile, SOURCES))
        native.result()
    objs = [o for o, _ in results]
    with open(os.path.join(OUT_DIR, "ptxas.txt"), "w") as f:
        for (o, log), src in zip(results, SOURCES):
            f.write(f"==== {src}\n{log}\n")
    check_registers(results[SOURCES.index("fa_fwd.cu")][1])
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(open(os.path.join(OUT_DIR, "ptxas.txt")).read(), file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
