"""Build the HIP libraries (kernels + C ABI) in-tree for gfx950: libgemm_rs.so
(the fused layer) and libgemm_rs_layer.so (the operators around it).

Run as ``python -m tensor_gemm_reduce_amd.build``.  hipcc cross-compiles the
device code for gfx950 without a GPU present.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_LAYER = os.path.join(PKG, "csrc_layer")
INCLUDE = os.path.join(ROOT, "include")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"


def library_path() -> str:
    return os.path.join(PKG, "libgemm_rs.so")


def layer_library_path() -> str:
    return os.path.join(PKG, "libgemm_rs_layer.so")


def sources():
    return [os.path.join(CSRC, "gemm_rs.hip")]


def layer_sources():
    return [os.path.join(CSRC_LAYER, n) for n in ("w4.hip", "block_norm.hip", "checkpoint.hip", "route.hip", "fp8.hip")]


def compile_flags(csrc=CSRC):
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        # keep hand-free of packed FP32 instructions (v_pk_*_f32)
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-ffp-contract=off", "-Wall", "-Wno-unused-function",
        "-I", INCLUDE, "-I", csrc,
    ]


def _run(cmds, verbose):
    """Runs the commands side by side; raises with the compiler's messages if one fails."""
    procs = []
    for cmd in cmds:
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    texts = [p.communicate()[0] for p in procs]
    for p, text in zip(procs, texts):
        msgs = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if p.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs))


def build(verbose: bool = False, extra=()) -> str:
    """Compiles both libraries and returns the fused layer's path."""
    out, layer = library_path(), layer_library_path()
    tag = ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in layer_sources()]
        _run([[HIPCC, *compile_flags(), "-shared", *extra, "-o", out + tag, *sources()]]
             + [[HIPCC, *compile_flags(CSRC_LAYER), *extra, "-c", "-o", o, src]
                for o, src in zip(objs, layer_sources())], verbose)
        _run([[HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", layer + tag, *objs]], verbose)
    os.replace(out + tag, out)
    os.replace(layer + tag, layer)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
