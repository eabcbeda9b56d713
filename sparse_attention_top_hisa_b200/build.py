"""Build libhisa.so (the C-ABI CUDA library) in-tree for sm_100a.

Each .cu file under csrc/ is compiled by nvcc into an object with
``-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` and the objects are
linked into ``sparse_attention_top_hisa_b200/libhisa.so`` (CUDA runtime linked
statically).  csrc/torch_binding.cpp is compiled by g++ against the installed torch
into ``_hisa_torch.so``.  Run ``python -m sparse_attention_top_hisa_b200.build``.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhisa.so")
BINDING = os.path.join(HERE, "_hisa_torch.so")
BINDING_STAMP = os.path.join(OUT_DIR, "_hisa_torch.stamp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files.append(os.path.join(ROOT, "include", "hisa.h"))
    return files


def _compile(src: str, extra) -> str:
    obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
           "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj, *extra]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def binding_tag() -> str:
    """What the binding is compiled against: it reads the fields of torch's tensors itself."""
    import torch
    return (f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}, "
            f"c++11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def build_binding(force: bool = False) -> str:
    """Compile the argument checks of the per-step entry points; returns the module's path.  It
    is built again when its sources, the flags or what it is compiled against have changed."""
    src, header = os.path.join(CSRC, "torch_binding.cpp"), os.path.join(ROOT, "include", "hisa.h")
    newest = max(os.path.getmtime(f) for f in (src, header))
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"]
    tag = binding_tag()
    stamp = "\n".join([tag, *flags])
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest:
        try:
            with open(BINDING_STAMP) as f:
                if f.read() == stamp:
                    return BINDING
        except OSError:
            pass
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    inc = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", *flags, f'-DHISA_BUILT_FOR="{tag}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in inc), src, "-o", tmp, "-L" + os.path.join(base, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(OUT_DIR, exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(stamp)
    return BINDING


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every kernel source and link libhisa.so, and the binding; returns the
    library's path."""
    build_binding(force)
    srcs = sources()
    newest = max(os.path.getmtime(f) for f in _deps())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas" in sys.argv))
