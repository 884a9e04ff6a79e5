"""Build libq8kv.so (the CUDA library behind include/q8kv.h) in-tree for sm_100a, and the compiled
half of its torch binding."""
from __future__ import annotations

import contextlib
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libq8kv.so")
MAIN_SRC = os.path.join(CSRC, "q8kv_api.cu")
BINDING = os.path.join(PKG, "_q8kv_torch.so")
BINDING_SRC = os.path.join(PKG, "binding", "q8kv_torch.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the q8kv CUDA library cannot be built")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "q8kv.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/q8kv_api.cu into decode_attention_int8_b200/libq8kv.so if stale."""
    if not force and not stale():
        return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, MAIN_SRC, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def binding_command(out: str) -> list:
    """The compile command of the binding, against the running torch and Python."""
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return [
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
        "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(cuda, "include"),
        "-isystem", sysconfig.get_paths()["include"],
        BINDING_SRC, "-o", out, "-L", os.path.join(torch_dir, "lib"),
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build_binding(force: bool = False) -> str:
    """Compile binding/q8kv_torch.cpp against the running torch if the module is stale: older than
    its sources, or built against another torch, Python or by another command (the record of
    that lies beside the module: one built against another torch may load, and read tensors by
    an outdated layout)."""
    import torch

    record = BINDING + ".built"
    # (of the command the flags: the folders may differ from one machine to the next)
    flags = [f for f in binding_command(BINDING) if not os.path.isabs(f)]
    against = "\n".join([torch.__version__, str(sysconfig.get_config_var("EXT_SUFFIX")), *flags])
    deps = [BINDING_SRC, os.path.join(INCLUDE, "q8kv.h")]
    if not force and os.path.exists(BINDING) and os.path.exists(record) and \
            all(os.path.getmtime(BINDING) >= os.path.getmtime(d) for d in deps):
        with open(record) as f:
            if f.read() == against:
                return BINDING
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.check_call(binding_command(tmp))
    with contextlib.suppress(FileNotFoundError):  # (never the old record beside a new module)
        os.remove(record)
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(against)
    os.replace(tmp, record)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_binding(force="--force" in sys.argv))
