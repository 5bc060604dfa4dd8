"""Builds libctcpb.so (the HIP decoder and its C ABI) and libctcpb_lm.so (the
language-model operators and theirs) for gfx950 with hipcc."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "ctcpb.hip")
LIB = os.path.join(HERE, "libctcpb.so")
LM_SRC = os.path.join(HERE, "csrc", "lm", "lm.hip")
LM_LIB = os.path.join(HERE, "libctcpb_lm.so")

# -ffp-contract=off: every float operation rounds once (the decoder's numerics
# are a fixed operation sequence).  Packed-FP32 instructions are disabled.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I" + os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function"]


# The language-model operators fix no operation sequence: products and sums may
# be contracted.
LM_FLAGS = [f for f in FLAGS if f != "-ffp-contract=off"]


def _compile(flags, src: str, lib: str, verbose: bool) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = lib + ".tmp"
    proc = subprocess.run([hipcc, *flags, src, "-o", tmp], capture_output=True, text=True)
    out = "\n".join(l for l in (proc.stdout + proc.stderr).splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out.strip():
        print(out)
    os.replace(tmp, lib)
    return lib


def build(verbose: bool = False) -> str:
    lib = _compile(FLAGS, SRC, LIB, verbose)
    build_lm(verbose)
    return lib


def build_lm(verbose: bool = False) -> str:
    return _compile(LM_FLAGS, LM_SRC, LM_LIB, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
