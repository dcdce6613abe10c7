"""Build libssm.so, libssm_block.so and libssm_delta.so (the HIP kernels and the
C ABIs) in-tree for gfx950.

    python -m state_space_model_ssm_amd.build

Each ``csrc/*.hip`` file is compiled with hipcc into ``_build/`` and linked
into ``state_space_model_ssm_amd/libssm.so``; ``csrc/block/*.hip`` go into
``libssm_block.so`` and ``csrc/delta/*.hip`` into ``libssm_delta.so`` alike.  Packed-FP32 instructions are disabled for all
device code.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssm.so")
BLOCK_CSRC = os.path.join(CSRC, "block")
BLOCK_LIB = os.path.join(PKG, "libssm_block.so")
DELTA_CSRC = os.path.join(CSRC, "delta")
DELTA_LIB = os.path.join(PKG, "libssm_delta.so")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}", f"-I{CSRC}",
]
# libssm_delta's matrix products leave their results in ordinary registers: in
# the accumulators, half of a recurrence's instructions were moves from and to them.
DELTA_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form"]


def _object(src: str) -> str:
    return os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")


def sources(folder: str = CSRC) -> list[str]:
    return sorted(os.path.join(folder, f) for f in os.listdir(folder) if f.endswith(".hip"))


def build(verbose: bool = False) -> str:
    """Compile every source and link the libraries. Returns libssm's path."""
    os.makedirs(BUILD, exist_ok=True)
    objects = {LIB: sources(), BLOCK_LIB: sources(BLOCK_CSRC), DELTA_LIB: sources(DELTA_CSRC)}
    procs = []
    for src in [src for srcs in objects.values() for src in srcs]:
        obj = _object(src)
        cmd = [HIPCC, *CFLAGS, *(DELTA_FLAGS if src in objects[DELTA_LIB] else []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        text = "\n".join(l for l in out.decode(errors="replace").splitlines()
                         if "is not a recognized feature" not in l)
        if pr.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        for src, text in failed:
            print(f"--- {src}\n{text}", file=sys.stderr)
        raise RuntimeError("hipcc failed for: " + ", ".join(os.path.basename(s) for s, _ in failed))
    for lib, srcs in objects.items():
        tmp = lib + ".tmp"
        link = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *map(_object, srcs), "-o", tmp]
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.check_call(link)
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
