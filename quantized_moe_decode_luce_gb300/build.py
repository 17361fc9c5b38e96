"""Build libluce_moe.so in-tree with nvcc for sm_103a (GB300), and beside it the
module that makes the common calls of the int8 head (g++, torch's headers),
which is an addition: without it every call goes through binding.py.

The translation units are compiled in parallel and linked into
``quantized_moe_decode_luce_gb300/lib/libluce_moe.so``.  Release flags only:
no fast-math (the quantization and the combine depend on IEEE division and
on separately rounded products and sums).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(LIBDIR, "libluce_moe.so")
SOURCES = ["small_ops.cu", "glu_pair.cu", "down_combine.cu", "moe_layer.cu", "moe_layer_flat.cu", "edge_ops.cu",
           "q4k_ops.cu", "moe_tc.cu", "rows_i8.cu", "linear_i8.cu", "logits_process.cu", "rows_w4.cu", "linear_w4.cu", "linear_w4_tc.cu",
           "sample.cu"]
CALL_SOURCE = "fastcall.cpp"
HEADERS = ["common.cuh", "w4.cuh", os.path.join("..", "..", "include", "luce_moe.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


# Sources whose warpgroups trade registers: a kernel there is launched with as many a thread as the first pattern finds in
# the source for the template argument that stands first in its name (the last two of the four modes take the second).
TRADING = {"linear_w4_tc.cu": (r"LAUNCH = RAW \? (\d+) : (\d+)", r"k_linear_w4_tcILi(\d)E")}


def check_registers(src: str, text: str, log: str) -> None:
    """Raises where the compiler gave a kernel of `src` fewer registers a thread (`log` is what -Xptxas -v printed) than
    its warpgroups share out (`text` is the source): the library would refuse to launch it."""
    share, entry = TRADING[src]
    needs = [int(n) for n in re.search(share, text).groups()]
    seen = re.findall(r"Compiling entry function '([^']*)'.*?Used (\d+) registers", log, re.S)
    modes = [(name, re.search(entry, name), int(regs)) for name, regs in seen]
    if not any(m for _, m, _ in modes):
        raise RuntimeError(f"{src}: the compiler told no kernel's registers")
    for name, m, regs in modes:
        if m and regs < needs[int(m.group(1)) // 2]:
            raise RuntimeError(f"{src}: {name} has {regs} registers a thread, its warpgroups share {needs[int(m.group(1)) // 2]}")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def call_path() -> str:
    """The call module of this Python and this torch: it is tied to both, so both stand in its name."""
    import torch
    version = re.sub(r"[^0-9A-Za-z.]+", "_", torch.__version__)
    return os.path.join(LIBDIR, f"luce_call.{sys.implementation.cache_tag}.torch-{version}.so")


def call_command(source: str, target: str) -> list[str]:
    """The g++ command for the call module, against this Python and this torch."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(root, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in inc), source,
            "-o", target, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libluce_moe.so."""
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers + [__file__]):
            jobs.append((src, s, o))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compilation failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return r

    def compile_one(job):
        src, s, o = job
        if src not in TRADING:
            return run([nvcc(), *ARCH, *NVCC_FLAGS, "-c", s, "-o", o])
        tmp = o + f".tmp{os.getpid()}.o"
        r = run([nvcc(), *ARCH, *NVCC_FLAGS, "-Xptxas", "-v", "-c", s, "-o", tmp])
        with open(s) as f:
            check_registers(src, f.read(), r.stderr + r.stdout)
        os.replace(tmp, o)

    def build_call():
        # (no torch, no headers, no compiler: the library does without the module)
        target = None
        try:
            target = call_path()
            source = os.path.join(CSRC, CALL_SOURCE)
            if force or _stale(target, [source, headers[-1], __file__]):
                tmp = target + f".tmp{os.getpid()}"
                run(call_command(source, tmp))
                os.replace(tmp, target)
        except (ImportError, OSError, RuntimeError) as e:
            if target is not None and os.path.exists(target):
                os.remove(target)  # one of an older source
            warnings.warn(f"the call module is not built, calls of the int8 head go through binding.py: {e}",
                          RuntimeWarning, stacklevel=2)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call = ex.submit(build_call)
        list(ex.map(compile_one, jobs))
        call.result()
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
