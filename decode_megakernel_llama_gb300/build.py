"""Builds libmk.so (the megakernel and its C ABI) in-tree for sm_103a, and mk_torch, the binding's extension module."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmk.so")
LIB_CHECKED = os.path.join(BUILD, "libmk_checked.so")
SOURCES = ["mk_kernel_hd64.cu", "mk_kernel_hd128.cu", "mk_kernel.cu", "mk_host.cpp", "mk_noalloc.cu", "mk_w2a8.cu",
           "mk_prefill.cu", "mk_twell.cu"]
DEPS = SOURCES + ["mk_kernel.cuh", "mk_plan.h", "mk_internal.h", "mk_prefill.h"]
# the standalone operators: units of their own beside the megakernel's, and the
# extension module through which the binding calls them with torch's tensors
OP_SOURCES = ["mk_rope.cu", "mk_tree.cu", "mk_kv.cu"]
OP_DEPS = OP_SOURCES + ["mk_ops.h", "mk_tc.cuh", "mk_tree_attn.cuh"]
TORCH_SOURCE = "mk_torch.cpp"


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmk.so")


def flags() -> list[str]:
    return ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", f"-I{os.path.join(ROOT, 'include')}"]


def extension_path() -> str:
    """The extension module for the torch and Python that run this: it unpacks torch's objects, so another torch's
    or Python's is another file."""
    import sys

    import torch
    return os.path.join(BUILD, f"mk_torch.{sys.implementation.cache_tag}.torch-{torch.__version__}."
                               f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}.so")


def torch_command(out: str) -> list[str]:
    """The compiler's command for the extension module, against the torch and Python that run this."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in inc],
            os.path.join(CSRC, TORCH_SOURCE), "-o", out, f"-L{os.path.join(root, 'lib')}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _stale(lib: str, sources: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, s) for s in sources] + [os.path.join(ROOT, "include", "mk.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """checked=True builds libmk_checked.so: every device-side access is
    validated against the registered buffers (slow; for diagnosing faults).

    The library needs neither torch nor Python's headers: without torch it is built
    alone, and where the extension module does not compile it is there before that is
    raised."""
    lib = LIB_CHECKED if checked else LIB
    os.makedirs(BUILD, exist_ok=True)
    try:
        ext = extension_path()
    except ImportError:
        ext = None  # (no torch: nothing that the extension module could serve)
    ext_proc = None
    if ext and (force or _stale(ext, [TORCH_SOURCE])):
        ext_tmp = ext + f".tmp{os.getpid()}"
        ext_cmd = torch_command(ext_tmp)
        ext_proc = subprocess.Popen(ext_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    try:
        if force or _stale(lib, DEPS + OP_DEPS):
            _build_lib(lib, verbose, checked)
    finally:
        if ext_proc is not None:
            out, _ = ext_proc.communicate()
    if ext_proc is not None:
        if ext_proc.returncode:
            print(out.decode(errors="replace"))
            raise RuntimeError(f"compile failed: {' '.join(ext_cmd)}")
        os.replace(ext_tmp, ext)
    return lib


def _build_lib(lib: str, verbose: bool, checked: bool) -> None:
    nv = nvcc()
    procs, objs = [], []
    tag = ".chk" if checked else ""
    for s in SOURCES + OP_SOURCES:
        obj = os.path.join(BUILD, s + tag + ".o")
        extra = ["-Xptxas", "-v"] if (verbose and s.endswith(".cu")) else []
        if checked:
            extra += ["-DMK_CHECKED"]
        cmd = [nv, *flags(), *extra, "-c", os.path.join(CSRC, s), "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    for cmd, pr in procs:
        out, _ = pr.communicate()
        if verbose or pr.returncode:
            print(out.decode(errors="replace"))
        if pr.returncode:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}")
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nv, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp, *objs],
                   check=True)
    os.replace(tmp, lib)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                checked="--checked" in sys.argv))
