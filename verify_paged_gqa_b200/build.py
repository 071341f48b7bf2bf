"""Builds libtfpaged.so (the C-ABI CUDA library) in place, for sm_100a only, and
_binding.so (torch tensors to that ABI) beside it.

    python -m verify_paged_gqa_b200.build [--verbose]

nvcc compiles each translation unit under csrc/ to an object in _build/ and
links them into verify_paged_gqa_b200/libtfpaged.so.  ``--verbose`` adds
``-Xptxas -v`` (registers, spills, shared memory per kernel) to the log.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build", "tfpaged")
LIB = os.path.join(HERE, "libtfpaged.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(HERE, "_binding.so.for")   # the Python and torch it was compiled against
SOURCES = ["tf_paged.cu", "kv_put.cu", "kv_rope.cu", "kv_copy.cu", "kv_pages.cu", "attn_simt.cu", "attn_win.cu",
           "attn_prompt.cu", "attn_pm.cu", "attn_merge.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA library cannot be built")
    return cand


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "tf_paged.h"))
    return files


def _newer_than_sources(path) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _deps())


def _interpreter() -> str:
    """What _binding.so is compiled against: it loads under no other Python or torch."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__}"


def _binding_up_to_date() -> bool:
    if not _newer_than_sources(BINDING) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == _interpreter()


def up_to_date() -> bool:
    return _newer_than_sources(LIB) and _binding_up_to_date()


# host-compiler flags of the sanitizer build (one per -Xcompiler: nvcc splits
# an -Xcompiler value at commas)
SANITIZE = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
            "-fno-omit-frame-pointer"]


def build_binding() -> None:
    """Compile csrc/binding.cpp against the running interpreter's torch."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(_interpreter())
    os.replace(tmp, BINDING_FOR)


def build(verbose: bool = False, force: bool = False, sanitize: bool = False) -> str:
    """Compile and link the library; returns its path.  ``sanitize`` builds a
    separate copy (_build/asan/libtfpaged_asan.so) whose host code carries
    AddressSanitizer and UndefinedBehaviorSanitizer (device code is
    unchanged; the process that loads it must preload libasan)."""
    if not sanitize and not force and not verbose and _newer_than_sources(LIB):
        if not _binding_up_to_date():
            build_binding()
        return LIB
    build_dir = os.path.join(ROOT, "_build", "asan") if sanitize else BUILD
    lib = os.path.join(build_dir, "libtfpaged_asan.so") if sanitize else LIB
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []
    if sanitize:
        extra += [f"-Xcompiler={f}" for f in SANITIZE] + ["-g"]

    def compile_one(src):
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if sanitize else ex.submit(build_binding)
        results = list(ex.map(compile_one, SOURCES))
    log = "".join(out for _, out in results)
    with open(os.path.join(build_dir, "ptxas.log"), "w") as f:
        f.write(log)
    tmp = lib + f".tmp{os.getpid()}"
    link_extra = ["-Xcompiler=-fsanitize=address", "-Xcompiler=-fsanitize=undefined"] if sanitize else []
    cmd = [cc, *ARCH, "-shared", *link_extra, "-o", tmp, *[o for o, _ in results], "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if verbose:
        sys.stdout.write(log)
    if binding is not None:
        binding.result()   # (the library is there whether or not it compiled)
    return lib


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
