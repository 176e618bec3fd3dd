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


def kernels(call, plan, cus=256):
    """The kernels that a call with this plan launches, as (name, template
    arguments but the type)."""
    kind, p, out = call[0], plan, set()
    if kind == "tn":
        groups, sums, layout = call[4] > 0, bool(call[5]), 2
    else:
        groups, sums, layout = kind == "grouped", False, call[1]
    if p.tile_m < 128:
        out.add(("gemm_small", layout, p.tile_m // 16, p.tile_n // 16, True, groups))
    else:
        tasks = p.tiles - p.split_tiles + p.split_tiles * p.parts
        deep = p.tile_m == p.tile_n == 128 and tasks <= cus and kind != "grouped"
        out.add(("layer_gemm_kernel", layout, p.parts > 1 or deep, p.tile_n, p.tile_m, groups, sums))
        if p.parts > 1:
            wide = p.split_tiles * p.tile_m * p.tile_n // (8 * 256) >= cus
            out.add(("split_reduce", p.tile_n, 256 if wide else 64, p.tile_m, True))
        elif p.sums_bytes:
            out.add(("column_sums", p.tile_m))
    if p.copies:
        out.add(("repack_groups",))
    return out


def traits(call, plan, cus=256):
    """What else a test of that kernel should meet: a workgroup that computes
    more than one tile, a last wave of tiles in parts, column sums with or
    without a second kernel."""
    p, out = plan, set()
    if p.tile_m >= 128:
        slots = cus * (2 if p.tile_m == p.tile_n == 128 else 1)
        tiles = p.tiles
        if call[0] == "grouped":  # (however the rows are shared out)
            tiles = -(-call[2] // p.tile_m) * -(-call[3] // p.tile_n)
        if tiles > slots:
            out.add("more than one round")
        if 0 < p.split_tiles < p.tiles:
            out.add("last wave in parts")
    if call[0] == "tn" and call[5]:
        out.add("partial column sums" if p.sums_bytes else "column sums in the first tiles")
    return frozenset(out)
