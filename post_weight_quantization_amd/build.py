"""Build libgptq_mi355x.so in-tree with hipcc for gfx950 (every call recompiles)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgptq_mi355x.so")
SOURCES = ["fold.hip", "fold64.hip", "sweep.hip", "gram.hip", "debias.hip", "act_order.hip", "api.hip",
           "check.hip", "round.hip", "linear.hip", "cache.hip", "attention.hip"]
ARCH = "gfx950"
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-ffp-contract=fast-honor-pragmas", "-fno-gpu-rdc",
         # The sweep's column loops are sized for the unroller before their lane broadcasts fold
         # to single DPP moves; left rolled, each broadcast becomes a branch tree.
         "-mllvm", "-pragma-unroll-threshold=200000",
         "-Rpass-analysis=kernel-resource-usage"]  # remarks only: see SPILLS

# Vector registers that kernels may spill: instances whose variants without are slower (measured, at the
# kernels).  Template arguments as they are mangled: type (0 f32, 1 bf16, 2 f16) and dim / 32.
SPILLS = {"attention_tile_kernelILi0ELi8EE": 28, "attention_tile_kernelILi1ELi4EE": 1,
          "attention_tile_kernelILi1ELi8EE": 19, "attention_tile_kernelILi2ELi4EE": 27}


def spills(remarks: str) -> dict:
    """Kernels of the compiler's resource remarks that spill vector registers: {mangled name: registers}."""
    found, name = {}, None
    for line in remarks.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name = m.group(1)
        m = re.search(r"VGPRs Spill: (\d+)", line)
        if m and int(m.group(1)):
            found[name] = int(m.group(1))
    return found


def too_many(found: dict) -> list:
    """Those of the spilling kernels that SPILLS does not allow for."""
    return [f"{name} spills {n} vector registers" for name, n in found.items()
            if n > max((v for k, v in SPILLS.items() if k in name), default=0)]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = ["hipcc", *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    # Every unroll pragma must take effect (a build error rather than a slow kernel).
    if "loop not unrolled" in r.stderr:
        raise RuntimeError(f"hipcc left a loop rolled in {src}:\n{r.stderr}")
    over = too_many(spills(r.stderr))
    if over:
        raise RuntimeError(f"{src}: " + "; ".join(over))
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = ["hipcc", "-shared", f"--offload-arch={ARCH}", "-fPIC", "-pthread", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
