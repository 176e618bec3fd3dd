"""The plans of the layer products for 256 CUs, on the CPU."""
import re
import shutil
import subprocess

import pytest

from dense_gemm_08_amd import binding
from tests import _layer_cases, _plans
from tests._plans import NN, NT

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


def tile(*call):
    p = _plans.plans([call])[0]
    return p.tile_m, p.tile_n


def test_rounds_of_tiles_are_counted_for_outputs_of_one_tile_row_or_column():
    # 128-row (A @ B.T: or 128-column) tiles that take more than one round:
    # costed as one they were taken where 128 x 128 tiles are faster (measured:
    # 128 x 200000 x 512 79 against 64 us, 150000 x 64 x 256 41 against 27)
    for layout in (NT, NN):
        for M, N, K in ((128, 200000, 512), (100, 150000, 256), (128, 70000, 1024), (20, 100000, 1024)):
            assert tile("layer", layout, M, N, K) == (128, 128)
        # they stay over a long K
        assert tile("layer", layout, 128, 200000, 4096) == (128, 256)
    assert tile("layer", NT, 200000, 128, 512) == (128, 128)
    assert tile("layer", NT, 150000, 64, 256) == (128, 128)
    assert tile("layer", NT, 200000, 128, 4096) == (256, 128)


def compiled():
    """The instantiations of the layer kernels in the library, as _plans.kernels
    names them (FP16's; the types share the templates)."""
    names = subprocess.run(["nm", binding.library_path()], capture_output=True, text=True, check=True).stdout
    out = set()
    for name, args in re.findall(r"__device_stub__(layer_gemm_kernel|gemm_small|column_sums)I((?:DF16_|L[ib]\d+E)+)E",
                                 names):
        if args.startswith("DF16_"):
            values = re.findall(r"L([ib])(\d+)E", args)
            out.add((name,) + tuple(bool(int(v)) if t == "b" else int(v) for t, v in values))
    return {k for k in out if k[0] != "gemm_small" or k[4]}  # (the layer's form)


def reached():
    ps = _plans.plans(_layer_cases.CALLS)
    return [(k, _plans.traits(c, p)) for c, p in zip(_layer_cases.CALLS, ps) for k in _plans.kernels(c, p)]


@pytest.mark.skipif(shutil.which("nm") is None, reason="nm not available")
def test_every_compiled_kernel_is_reached_by_a_call():
    have, met = compiled(), {k for k, _ in reached()}
    assert len(have) > 40
    assert not have - met, sorted(have - met)
    assert not {k for k in met if k[0] in ("layer_gemm_kernel", "gemm_small", "column_sums")} - have


def test_the_listed_calls_meet_the_second_tile_and_the_last_wave():
    """Where a workgroup's second tile follows its first, and where whole tiles
    and parts share a launch, each kernel that can come to it does."""
    met = {}
    for kernel, traits in reached():
        met.setdefault(kernel, []).append(traits)
    for kernel, seen in met.items():
        if kernel[0] != "layer_gemm_kernel":
            continue
        _, layout, split, tn, tm, groups, sums = kernel
        if not split:
            assert any("more than one round" in t for t in seen), kernel
        elif tn == tm == 256 and not groups:
            assert any("last wave in parts" in t for t in seen), kernel
            assert any("last wave in parts" not in t for t in seen), kernel
        if sums:
            assert any("partial column sums" in t for t in seen), kernel
            if not (split and tm == 256):  # (a split 256 x 256 tile has a long K)
                assert any("column sums in the first tiles" in t for t in seen), kernel
    # the sums of whole tiles and of a last wave's parts, added up together
    assert any({"last wave in parts", "partial column sums"} <= t for ts in met.values() for t in ts)
    # the reduction with one-wave and with 256-thread workgroups, and each tile
    reductions = {k[1:4] for k in met if k[0] == "split_reduce"}
    assert {(128, 64, 128), (128, 256, 128), (128, 256, 256), (256, 256, 128), (256, 64, 256),
            (256, 256, 256)} <= reductions
