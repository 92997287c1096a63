"""Build libkpool.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m pool_score_top_amd.build        # or __graft_entry__.build()

hipcc cross-compiles the device code for gfx950; no GPU is needed.  Packed
fp32 instructions are disabled for all device code.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkpool.so")
# (layer.hip includes api.hip: one translation unit with the C ABI's shared state)
SOURCES = ["layer.hip", "pool_keys.hip", "score.hip", "topk.hip", "expand.hip", "norm.hip",
           "rotary.hip", "attend.hip", "attend_bwd.hip", "latent.hip"]
# Per-file flags.  The score kernel runs with the IEEE mode bit off so that the
# ReLU is one v_max_f32 (no NaN-quieting canonicalize before it); its inputs are
# finite bf16 / fp32 values, and NaN propagation is the only behaviour this changes.
# (Its instruction order is pinned in the source with scheduling-group barriers; the
# max-ILP machine scheduler measured ~2% slower with them than the default one.)
# The latent attention's kernels hold up to 500 registers: results of matrix instructions stay in
# ordinary registers (vector instructions cannot take accumulation registers, and copies to and fro
# would double them), the queries' fragments in accumulation registers.
FILE_FLAGS = {"score.hip": ["-mno-amdgpu-ieee", "-fno-honor-nans"],
              "latent.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                     if "packed-fp32-ops" not in l and "--hip-link" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{' '.join(cmd)}\n{msgs}")
    if verbose and msgs.strip():
        print(msgs)


def build(verbose: bool = False, extra=()) -> str:
    """Compile every source to an object (in parallel), then link libkpool.so."""
    from concurrent.futures import ThreadPoolExecutor
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    compile_flags = [f for f in FLAGS if f != "-shared"]
    jobs = []
    for s in SOURCES:
        obj = os.path.join(objdir, s.replace(".hip", ".o"))
        jobs.append(([HIPCC, *compile_flags, *FILE_FLAGS.get(s, []), *extra, "-c",
                      os.path.join(CSRC, s), "-o", obj], obj))
    with ThreadPoolExecutor(len(jobs)) as ex:
        list(ex.map(lambda j: _run(j[0], verbose), jobs))
    tmp = LIB + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *[o for _, o in jobs]], verbose)
    os.replace(tmp, LIB)
    build_example(verbose)
    return LIB


EXAMPLE_SRC = os.path.join(HERE, "examples", "select_file.c")
EXAMPLE = os.path.join(HERE, "examples", "select_file")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def build_example(verbose: bool = False) -> str:
    """The C example (a plain C99 host program over the C ABI and the HIP runtime),
    built with the system C compiler against the library next to it."""
    tmp = EXAMPLE + ".tmp"
    _run(["gcc", "-std=c99", "-O2", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
          f"-I{ROCM}/include", EXAMPLE_SRC, "-o", tmp, f"-L{HERE}", "-lkpool", f"-L{ROCM}/lib",
          "-lamdhip64", "-lm", "-Wl,-rpath,$ORIGIN/..", f"-Wl,-rpath,{ROCM}/lib"], verbose)
    os.replace(tmp, EXAMPLE)
    return EXAMPLE


if __name__ == "__main__":
    print(build(verbose=True, extra=sys.argv[1:]))
