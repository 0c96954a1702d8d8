"""Build the HIP library ``libmoe_lora.so`` for gfx950 with hipcc.

Every ``csrc/*.hip`` file is compiled to an object (in parallel), then linked
into one shared library next to this file, for which hipcc is all it takes.
``csrc/operands.c``, the binding's look at its tensors, becomes the extension
module ``_operands`` where torch, Python's headers and a C compiler are there:
without it the library is whole for its other users, and the calls that need the
module say so.  Always rebuilds when called.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
SO = os.path.join(PKG, "libmoe_lora.so")
OPERANDS = os.path.join(PKG, "_operands.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    # no packed fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_operands() -> str:
    import torch
    # (not hipcc, which would link its HIP runtime beside torch's)
    cc = next((c for c in ("gcc", "cc", "clang", os.path.join(os.path.dirname(HIPCC), "amdclang")) if shutil.which(c)),
              None)
    if cc is None:
        raise RuntimeError("no C compiler for operands.c")
    tmp = OPERANDS + ".tmp%d" % os.getpid()
    r = subprocess.run([cc, "-O2", "-Wall", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I",
                        sysconfig.get_paths()["include"], "-I",
                        os.path.join(os.path.dirname(torch.__file__), "include"),
                        os.path.join(CSRC, "operands.c"), "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed for operands.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPERANDS)
    return OPERANDS


def build(jobs: int | None = None) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = SO + ".tmp%d" % os.getpid()
    r = subprocess.run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, SO)
    try:
        build_operands()
    except (ImportError, RuntimeError) as e:
        if os.path.exists(OPERANDS):
            os.remove(OPERANDS)  # none rather than an older one
        warnings.warn(f"{SO} is built, lora_moe_amd._operands is not: {e}")
    return SO


if __name__ == "__main__":
    print(build())
