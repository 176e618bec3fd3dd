"""The plans of the layer products for 256 CUs, on the CPU."""
import shutil

import pytest

from tests import _plans
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
