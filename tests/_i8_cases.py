"""Calls of the int8 products that between them launch every kernel of theirs on
256 CUs (tests/test_i8_plans.py sees to that; tests/test_gpu_i8.py runs them), and
their plans (csrc/plan_experts.cpp) from a host build."""
import os
import subprocess
import tempfile

from tests._plans import Plan

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

I8 = [  # M, N, K
    (1, 1, 1), (1, 1, 4), (16, 33, 300), (7, 4096, 4096), (1, 18256, 513), (30, 900, 260), (60, 2095, 1000),
    (64, 8192, 2048), (90, 4632, 401), (128, 16384, 516), (33, 2174, 8192), (100, 8000, 6000), (20, 70000, 300),
    (136, 400, 6), (300, 264, 9001), (512, 512, 8192), (777, 1001, 2051), (700, 521, 90), (1000, 8192, 128),
    (129, 129, 40000), (256, 128, 40004), (8192, 100, 20000), (100, 86000, 2200), (86000, 100, 2200),
    (65, 38167, 10826), (65, 90000, 10826), (2095, 4060, 1948), (4096, 4096, 512), (3000, 5000, 1000), (4787, 3756, 2200),
    (2000, 3000, 4096), (4352, 4096, 4096), (4000, 4100, 8192), (257, 300, 131071), (120, 256, 131071),
    (20, 20, 131071), (5000, 40, 64), (40, 5000, 64), (256, 256, 128), (512, 256, 16384), (300, 100, 50000),
    (300, 128, 8192), (2560, 3000, 20000), (137, 8909, 13776), (9645, 133, 14189), (33, 66563, 2239),
    (34, 70644, 2100),
]

GROUPED = [  # rows, N, K, groups
    (1, 1, 1, 1), (1, 1, 4, 3), (20, 300, 700, 4), (32, 2048, 2048, 64), (44, 10, 1, 1), (300, 33, 403, 100),
    (3001, 300, 203, 7), (5003, 1400, 1000, 48), (2048, 512, 4096, 4), (8192, 2048, 512, 64),
    (6000, 1000, 4096, 6), (4096, 4096, 1024, 16), (16384, 1024, 256, 16), (9000, 700, 130, 300),
    (5000, 4100, 4096, 16), (9001, 2050, 4098, 16),
]

_exe = None


def plans(lines, cus=256):
    global _exe
    if _exe is None:
        folder = tempfile.TemporaryDirectory(prefix="experts_plans")
        exe = os.path.join(folder.name, "experts_plans")
        csrc = os.path.join(ROOT, "dense_gemm_08_amd", "csrc")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(HERE, "experts_plans.cpp")] +
                       [os.path.join(csrc, n) for n in ("plan.cpp", "plan_layer.cpp", "plan_experts.cpp")] +
                       ["-o", exe], check=True)
        _exe = (exe, folder)  # (the directory lives as long as the process)
    text = "\n".join(" ".join(map(str, line)) for line in lines)
    r = subprocess.run([_exe[0], str(cus)], input=text + "\n", capture_output=True, text=True, check=True)
    return [Plan(*map(int, line.split())) for line in r.stdout.splitlines()]


def kernels(kind, p, cus=256):
    """The kernels that a call with this plan launches, as (name, template
    arguments but the type)."""
    out = set()
    if p.tile_m < 128:
        out.add(("gemm_small_i8", p.tile_m // 16, p.tile_n // 16, kind == "grouped"))
    else:
        tasks = p.tiles - p.split_tiles + p.split_tiles * p.parts
        deep = p.tile_m == p.tile_n == 128 and tasks <= cus and kind == "i8"
        out.add(("layer_gemm_kernel", 0, p.parts > 1 or deep, p.tile_n, p.tile_m, kind == "grouped", False))
        if p.parts > 1:
            out.add(("split_reduce_i8", p.tile_n, p.tile_m))
    if p.copies:
        out.add(("repack_i8",))
    return out
