"""Build libsrnl.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
# translation units, compiled side by side and linked into the one library
UNITS = [os.path.join(PKG, "csrc", "layers", f)
         for f in ("operator_unit.hip", "linear.hip", "narrow_bf16.hip", "narrow_fp32.hip",
                   "narrow_slope_bf16.hip", "narrow_slope_fp32.hip", "layers.hip", "group_norm.hip",
                   "dropout.hip", "delta.hip", "delta_step.hip", "delta_prep.hip", "delta_chain.hip",
                   "delta_grads.hip")]
LIB = os.path.join(PKG, "libsrnl.so")
# the same source with the scan kernel's phase clocks compiled in (a
# measurement build, loaded only by bench.py --phase-clocks)
PHASE_LIB = os.path.join(PKG, "libsrnl_phase.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-result",
    # no packed fp32 instructions (hipcc warns on the host pass: harmless)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA accumulators in ordinary VGPRs, so that the VALU work between
    # dependent products needs no accumulator-register copies
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-I", os.path.join(ROOT, "include"),
]


def build(verbose: bool = False, phase_clocks: bool = False) -> str:
    lib = PHASE_LIB if phase_clocks else LIB
    extra = ["-DSRNL_PHASE_CLOCKS=1"] if phase_clocks else []
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(u) + ".o") for u in UNITS]
        cmds = [[HIPCC] + FLAGS + extra + ["-c", "-o", o, u] for u, o in zip(UNITS, objs)]
        runs = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
            runs.append(subprocess.Popen(cmd))
        codes = [r.wait() for r in runs]
        for cmd, code in zip(cmds, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        out = lib + ".tmp"
        cmd = [HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", out] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    os.replace(out, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, phase_clocks="--phase-clocks" in sys.argv))
