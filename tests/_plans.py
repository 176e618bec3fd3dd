"""The layer products' plans (csrc/plan_layer.cpp), from a host build."""
import os
import subprocess
import tempfile
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NT, NN = 0, 1
Plan = namedtuple("Plan", "tile_m tile_n tiles parts split_tiles copies sums_bytes", defaults=(0,))
_exe = None


def program():
    global _exe
    if _exe is None:
        _dir = tempfile.TemporaryDirectory(prefix="layer_plans")
        exe = os.path.join(_dir.name, "layer_plans")
        csrc = os.path.join(ROOT, "dense_gemm_08_amd", "csrc")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "include"),
                        "-I", csrc, os.path.join(HERE, "layer_plans.cpp"), os.path.join(csrc, "plan.cpp"),
                        os.path.join(csrc, "plan_layer.cpp"), "-o", exe], check=True)
        _exe = (exe, _dir)  # (the directory lives as long as the process)
    return _exe[0]


def plans(lines, cus=256):
    """The plans of calls like ("layer", NT, M, N, K), ("grouped", NN, M, N, K,
    G) and ("tn", M, N, K, G, sums), G = 0 without groups."""
    text = "\n".join(" ".join(str(int(v) if not isinstance(v, str) else v) for v in line) for line in lines)
    r = subprocess.run([program(), str(cus)], input=text + "\n", capture_output=True, text=True, check=True)
    return [Plan(*map(int, line.split())) for line in r.stdout.splitlines()]
