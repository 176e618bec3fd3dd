"""The plans of the int8 products for 256 CUs, on the CPU."""
import re
import shutil
import subprocess

import pytest

from dense_gemm_08_amd import binding
from tests import _i8_cases

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or shutil.which("nm") is None,
                                reason="g++ or nm not available")


def compiled():
    """The instantiations for FP16 results in the library (the types share the
    templates), as _i8_cases.kernels names them."""
    names = subprocess.run(["nm", binding.library_path()], capture_output=True, text=True, check=True).stdout
    out = set()
    for name, args in re.findall(r"__device_stub__layer_gemm_kernelINS_2I8I(DF16_)EE((?:L[ib]\d+E)+)E", names):
        out.add(("layer_gemm_kernel",) + _values(args))
    for name, args in re.findall(r"__device_stub__(gemm_small_i8|split_reduce_i8)IDF16_((?:L[ib]\d+E)+)E", names):
        out.add((name,) + _values(args))
    return out


def _values(args):
    return tuple(bool(int(v)) if t == "b" else int(v) for t, v in re.findall(r"L([ib])(\d+)E", args))


def test_every_compiled_kernel_is_reached_by_a_listed_call():
    met = set()
    for kind, calls in (("i8", _i8_cases.I8), ("grouped", _i8_cases.GROUPED)):
        for p in _i8_cases.plans([(kind,) + c for c in calls]):
            met |= _i8_cases.kernels(kind, p)
    have = compiled()
    assert len(have) >= 18
    assert not have - met, sorted(have - met)
    assert not {k for k in met if k[0] != "repack_i8"} - have
    assert ("repack_i8",) in met


def test_tiles_of_groups():
    def tile(*call):
        return _i8_cases.plans([("grouped",) + call])[0].tile_m
    # measured faster in 256 x 256 tiles, and in 128 x 128 ones
    for call in ((4096, 4096, 4096, 16), (16384, 4096, 4096, 16), (16384, 2048, 4096, 32), (16384, 2048, 2048, 64)):
        assert tile(*call) == 256
    for call in ((2048, 512, 4096, 4), (14400, 1400, 2000, 48), (8192, 2048, 2048, 64)):
        assert tile(*call) == 128


def test_tiles_of_groups_follow_what_was_measured():
    # every shape whose two times stand beside the estimate, and the limits by rows
    # a group and by the number of tiles
    def tile(*call):
        return _i8_cases.plans([("grouped",) + call])[0].tile_m
    measured = {(4096, 4096, 4096, 16): 256, (16384, 4096, 4096, 16): 256, (16384, 4096, 2048, 16): 256,
                (16384, 2048, 4096, 32): 256, (16384, 2048, 2048, 64): 256, (2048, 512, 4096, 4): 128,
                (14400, 1400, 2000, 48): 128, (25600, 1024, 4096, 128): 256}
    for call, want in measured.items():
        assert tile(*call) == want, call
    for call in ((2048, 4096, 4096, 16), (8192, 2048, 2048, 64), (2560, 4096, 4096, 16), (12288, 2048, 2048, 64),
                 (20480, 1024, 4096, 128), (32, 2048, 2048, 32), (256, 2048, 2048, 32)):
        assert tile(*call) == 128, call
    for call in ((8, 4096, 4096, 8), (128, 4096, 4096, 8), (64, 2048, 2048, 16)):
        assert tile(*call) == 16, call


def test_tiles_of_one_matrix_are_the_16_bit_ones():
    shapes = ((8192, 8192, 1024), (8192, 8192, 1536), (8192, 8192, 1664), (4096, 4096, 1024), (16384, 4096, 1024),
              (5000, 5000, 1500), (3000, 5000, 1024))
    for s, p in zip(shapes, _i8_cases.plans([("i8",) + s for s in shapes])):
        assert (p.tile_m, p.tile_n, p.parts) == (128, 128, 1), s
    assert _i8_cases.plans([("i8", 4096, 4096, 2048)])[0].tile_m == 256
