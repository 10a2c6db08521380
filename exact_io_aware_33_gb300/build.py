"""Builds libfa.so in-tree with nvcc for sm_103a (GB300), and the paged cache's
Python binding with the host compiler.

Each translation unit under ``csrc/`` is compiled in parallel into
``_build/`` at the repository root and linked into ``libfa.so`` (and
``_paged_native.so``, which links against it and PyTorch) next to this file. A
unit is recompiled only when it, or a header it may include, is newer than its
object file; the binding also when Python or PyTorch is another one.

libfa.so needs nvcc alone. Where the binding cannot be built (no PyTorch, one
without CUDA, no g++), the library is built all the same, and the paged cache
says so when it is first used.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfa.so")
BINDING = os.path.join(PKG, "_paged_native.so")

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_bwd_noalloc.cu", "fa_paged_append.cu",
           "fa_paged_attn.cu", "fa_paged_chunk.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I" + INCLUDE, "-I" + CSRC] + ARCH


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is needed to build libfa.so")


def cxx() -> str:
    path = shutil.which("g++") or shutil.which("c++")
    if path:
        return path
    raise RuntimeError("g++ not found: the paged cache's binding is built with it")


def _headers():
    out = []
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".h", ".cuh")):
                out.append(os.path.join(d, f))
    return out


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _binding_stamp() -> str:
    """What the binding was built against: this Python and the PyTorch that it would import."""
    origin = importlib.util.find_spec("torch").origin or ""
    version = os.path.join(os.path.dirname(origin), "version.py")
    text = ""
    if os.path.exists(version):
        with open(version) as f:
            text = f.read()
    return "\n".join([sys.version, origin, text])


def _start_binding(args, which: int):
    """Starts g++ for the binding with its compile (0) or link (1) flags; the process, or why there is none."""
    try:
        return subprocess.Popen([cxx()] + args + _binding_flags()[which], stdout=subprocess.PIPE,
                                stderr=subprocess.STDOUT)
    except (RuntimeError, ImportError, OSError) as e:
        return str(e)


def _finish_binding(p) -> str:
    """Waits for what _start_binding gave; empty, or why it failed."""
    if p is None or isinstance(p, str):
        return p or ""
    out, _ = p.communicate()
    return "" if p.returncode == 0 else out.decode(errors="replace") or "g++ failed"


def _binding_flags():
    """(compile, link) flags of the binding: Python's and PyTorch's headers and libraries."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    flags = ["-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    link = ["-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG,
            "-l:libfa.so", "-Wl,-rpath,$ORIGIN"]
    return flags + ["-I" + i for i in include], link


def build(verbose: bool = False, force: bool = False, extra_flags=None, out_dir: str | None = None,
          lib_path: str | None = None) -> str:
    """Compile the CUDA sources and link libfa.so; returns the library path.

    ``out_dir`` / ``lib_path`` place the objects and the library elsewhere
    (used for test-only variants built with extra ``-D`` flags; the product
    library is always ``libfa.so`` next to this file)."""
    build_dir = out_dir or BUILD
    lib = lib_path or LIB
    os.makedirs(build_dir, exist_ok=True)
    exe = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    newest_header = max(os.path.getmtime(h) for h in _headers())
    procs, objs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(path), newest_header)):
            continue
        cmd = [exe, "-c", path, "-o", obj] + flags
        if verbose:
            cmd.append("-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    binding = compiling = None
    if lib == LIB and _has_torch():  # libfa.so itself needs no PyTorch
        path, binding = os.path.join(CSRC, "paged_binding.cpp"), os.path.join(build_dir, "paged_binding.o")
        stamp, stamp_file = _binding_stamp(), os.path.join(build_dir, "paged_binding.stamp")
        fresh = False
        if os.path.exists(stamp_file):
            with open(stamp_file) as f:
                fresh = f.read() == stamp
        if (force or not fresh or not os.path.exists(binding)
                or os.path.getmtime(binding) < max(os.path.getmtime(path), newest_header)):
            compiling = _start_binding(["-c", path, "-o", binding], 0)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    why = _finish_binding(compiling)  # there is no binding
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    if force or procs or not os.path.exists(lib) or any(
            os.path.getmtime(o) > os.path.getmtime(lib) for o in objs):
        tmp = lib + ".tmp"
        cmd = [exe, "-shared", "-o", tmp] + objs + ARCH
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, lib)
    if binding:
        if not why and (force or not fresh or not os.path.exists(BINDING)
                        or os.path.getmtime(BINDING) < max(os.path.getmtime(binding), os.path.getmtime(lib))):
            tmp = BINDING + ".tmp"
            why = _finish_binding(_start_binding(["-shared", "-o", tmp, binding], 1))
            if not why:
                os.replace(tmp, BINDING)
                with open(stamp_file, "w") as f:
                    f.write(stamp)
        if why:
            for old in (BINDING, stamp_file):  # one that is there does not fit what was built
                if os.path.exists(old):
                    os.remove(old)
            print(f"{lib} is built, the paged cache's Python binding is not:\n{why}", file=sys.stderr, flush=True)
    return lib


# Test-only variant for the bounded-wait (timeout) path: the forward's TMA
# producer never loads the last V tile of its key stream, and every wait gives
# up after 20 ms instead of about a second. It lives under _build/ and is
# never loaded by the package; only tests/test_timeout_path.py and
# tests/test_paged_timeout.py use it.
TIMEOUT_TEST_DIR = os.path.join(BUILD, "timeout_test")
TIMEOUT_TEST_FLAGS = ["-DFA_TEST_SKIP_ARRIVE", "-DFA_WAIT_BUDGET_NS=20000000ull"]


def build_timeout_test_variant(verbose: bool = False) -> str:
    """Build the test-only timeout variant of the library; returns its path."""
    return build(verbose=verbose, extra_flags=TIMEOUT_TEST_FLAGS, out_dir=TIMEOUT_TEST_DIR,
                 lib_path=os.path.join(TIMEOUT_TEST_DIR, "libfa_timeout_test.so"))


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
