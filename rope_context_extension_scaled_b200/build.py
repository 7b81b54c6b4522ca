"""Build librcx.so in-tree for sm_100a.

    python -m rope_context_extension_scaled_b200.build [--force] [-v]

Each csrc/*.cu file is one translation unit (the C-ABI host code, and one
unit per kernel family); they are compiled in parallel with nvcc and linked
into one shared library.  csrc/torch_binding.cpp becomes the extension module
_rcx_torch.so, which links to it and to the installed torch.
"""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
OUT = os.path.join(PKG, "librcx.so")
EXT_SRC = os.path.join(CSRC, "torch_binding.cpp")
EXT = os.path.join(PKG, "_rcx_torch.so")
EXT_ABI = os.path.join(OBJ, "_rcx_torch.abi")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [
    *ARCH,
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def units():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if not f.endswith((".cu", ".cpp"))] + \
        [os.path.join(ROOT, "include", "rcx.h")]


def _obj(src):
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    return _newest(units() + headers() + [os.path.abspath(__file__)]) <= os.path.getmtime(OUT)


def ext_abi() -> str:
    """What _rcx_torch.so is built against: another torch, Python or C++ ABI needs another build."""
    import torch
    return f"torch {torch.__version__}, cxx11 {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, python {sys.version}"


def ext_up_to_date() -> bool:
    deps = [EXT_SRC, os.path.join(ROOT, "include", "rcx.h"), os.path.abspath(__file__)]
    if not os.path.exists(EXT) or not os.path.exists(EXT_ABI) or _newest(deps) > os.path.getmtime(EXT):
        return False
    with open(EXT_ABI) as f:
        return f.read() == ext_abi()


def build_ext(force: bool = False) -> str:
    """Compile _rcx_torch.so against the installed torch (librcx.so has to be there)."""
    if not force and ext_up_to_date():
        return EXT
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-o", EXT + ".tmp",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in inc), EXT_SRC,
           "-L" + PKG, "-l:librcx.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("torch_binding.cpp failed:\n" + r.stdout + r.stderr)
    os.replace(EXT + ".tmp", EXT)
    os.makedirs(OBJ, exist_ok=True)
    with open(EXT_ABI, "w") as f:
        f.write(ext_abi())
    return EXT


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        build_ext()
        return OUT
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    hdr_time = _newest(headers() + [os.path.abspath(__file__)])
    procs = []
    for src in units():
        obj = _obj(src)
        if not force and os.path.exists(obj) and max(hdr_time, os.path.getmtime(src)) <= os.path.getmtime(obj):
            continue
        cmd = [nvcc, *NVCC_FLAGS, "-c", "-o", obj + ".tmp", src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, obj, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"{os.path.basename(src)}:\n{out}")
            continue
        if verbose:
            sys.stdout.write(out)
        os.replace(obj + ".tmp", obj)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    cmd = [nvcc, *ARCH, "-shared", "-o", OUT + ".tmp", *[_obj(s) for s in units()]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + r.stdout + r.stderr)
    os.replace(OUT + ".tmp", OUT)
    build_ext(force)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
