"""Build step for libdense_gemm.so (hipcc, gfx950 only).

``python -m dense_gemm_08_amd.build`` compiles ``csrc/plan.cpp``,
``csrc/plan_layer.cpp`` and ``csrc/plan_experts.cpp`` (host-side argument checks and launch planning, plain
C++), ``csrc/dense_gemm.hip`` (the FP16/BF16 entry points, kernels in
``gemm_kernel.h``), ``csrc/ladder.hip`` (the optimisation-step kernels),
``csrc/gemm_mx.hip`` (the FP8 block-scaled product, kernels in
``gemm_mx_kernel.h``), ``csrc/layer.hip``, ``csrc/grouped.hip`` and
``csrc/tn.hip`` (a layer's products and their gradients), ``csrc/i8.hip`` (the
same products in int8), ``csrc/route.hip`` (routing to experts) and
``csrc/rows.hip`` (rows quantised, and the experts' rows combined) into
``dense_gemm_08_amd/libdense_gemm.so`` in place.  The sources are compiled
side by side, then linked.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", n)
        for n in ("plan.cpp", "plan_layer.cpp", "plan_experts.cpp", "dense_gemm.hip", "ladder.hip",
                  "gemm_mx.hip", "layer.hip", "grouped.hip", "tn.hip", "i8.hip", "route.hip",
                  "rows.hip")]
OUT = os.path.join(HERE, "libdense_gemm.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # keep the compiler from forming packed FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]
JOBS = 6  # sources compiled at a time (each takes one core and under 1 GiB)


def build(extra=None, out=OUT, verbose=False) -> str:
    tmp = out + ".tmp%d" % os.getpid()
    compile_flags = [f for f in FLAGS if f != "-shared"] + list(extra or [])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory(prefix="dense_gemm_build") as objs:
        def compile_one(src):
            obj = os.path.join(objs, os.path.basename(src) + ".o")
            run([HIPCC] + compile_flags + ["-c", "-I", os.path.join(ROOT, "include"),
                                           "-I", os.path.join(HERE, "csrc"), src, "-o", obj])
            return obj

        with concurrent.futures.ThreadPoolExecutor(JOBS) as pool:
            made = list(pool.map(compile_one, SRCS))
        run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared"] + list(extra or []) + made +
            ["-o", tmp])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(extra=sys.argv[1:], verbose=True))
