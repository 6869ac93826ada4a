"""Build libswa_attn.so in-tree with nvcc for sm_103a, and the binding's
argument marshalling (csrc/marshal.cpp) with g++ against PyTorch's headers
(left out where PyTorch is not installed: the library needs none of it).

Each .cu under csrc/ is compiled to an object in parallel, then linked into
sliding_window_attention_gb300/libswa_attn.so.  Rebuilds only what changed
(sources and headers are compared by modification time).
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
SO = os.path.join(PKG, "libswa_attn.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libswa_attn.so")


MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))


MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")


def _torch_version():
    """The installed PyTorch's version, None without one."""
    if importlib.util.find_spec("torch") is None:
        return None
    import torch

    return torch.__version__


def _marshal_stamp() -> str:
    """The file that names the PyTorch that the module was built against."""
    return os.path.join(BUILD, os.path.basename(MARSHAL) + ".torch")


def _marshal_due(version, force: bool = False) -> bool:
    """Whether the module has to be built for this PyTorch."""
    if version is None:
        return False
    if force or not os.path.exists(MARSHAL) or not os.path.exists(_marshal_stamp()):
        return True
    with open(_marshal_stamp()) as f:
        if f.read() != version:
            return True
    return os.path.getmtime(MARSHAL) < max(os.path.getmtime(s) for s in (MARSHAL_SRC, os.path.join(ROOT, "include", "swa_attn.h")))


def _marshal_cmd(src: str, out: str):
    """g++ on the marshalling module.  The torch and CUDA symbols that it uses
    come from the libraries `import torch` has loaded."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", sysconfig.get_paths()["include"],
            "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, src, "-o", out,
            "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_mtime = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    procs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_mtime):
            continue
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    marshal_tmp = MARSHAL + f".tmp{os.getpid()}"
    torch_version = _torch_version()
    marshal_due = _marshal_due(torch_version, force)
    if marshal_due:
        cmd = _marshal_cmd(MARSHAL_SRC, marshal_tmp)
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((MARSHAL_SRC, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    if marshal_due:
        os.replace(marshal_tmp, MARSHAL)
        with open(_marshal_stamp(), "w") as f:
            f.write(torch_version)
    if force or not os.path.exists(SO) or any(os.path.getmtime(o) > os.path.getmtime(SO) for o in objs):
        tmp = SO + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
