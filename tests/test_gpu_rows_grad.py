"""What combine_rows_grad leaves where no place leads, on the GPU."""
import pytest

import dense_gemm_08_amd as dg
from tests import _experts
from tests.test_gpu_rows import choices, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def used_memory(shape, dtype):
    """Leaves a block of NaN with torch's allocator, for the next tensor of its
    size."""
    x = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,N,k,R,missing", [(3, 40, 2, 6, 0.5), (5, 1001, 3, 40, 0.0), (1, 8, 1, 1, 1.0),
                                             (300, 512, 2, 700, 0.2), (7, 4100, 4, 28, 0.3)])
def test_rows_that_no_place_names_are_zeros(T, N, k, R, missing, dtype):
    h, (p, w) = values(R, N, dtype), choices(T, k, R, missing=missing)
    p[p >= R] = -1
    dy = values(T, N, dtype, seed=1)
    print("combine_grad", T, N, k, R, dtype, flush=True)
    used_memory((R, N), h.dtype)
    dh, dw = dg.combine_rows_grad(dy, h, p, w)
    _experts.check_combine_grad(dh, dw, dy, h, p, w, torch.zeros_like(h), "no dh given")


def test_they_are_cleared_on_the_launch_stream():
    # (the current stream is still busy when the other one's kernels run)
    h, (p, w) = values(64, 300, "bf16"), choices(20, 2, 64, missing=0.3)
    p[p >= 64] = -1
    dy = values(20, 300, "bf16", seed=1)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        used_memory((64, 300), h.dtype)
        torch.cuda._sleep(20000000)
        dh, dw = dg.combine_rows_grad(dy, h, p, w, stream=stream)
        torch.cuda.synchronize()
        _experts.check_combine_grad(dh, dw, dy, h, p, w, torch.zeros_like(h), "on a stream")


def test_they_are_cleared_at_every_replay():
    h, dy = values(50, 136, "f16"), values(10, 136, "f16", seed=1)
    p, w = choices(10, 2, 50)
    p[p >= 50] = -1
    dg.combine_rows_grad(dy, h, p, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dh, dw = dg.combine_rows_grad(dy, h, p, w)
    for rep in range(4):
        q, _ = choices(10, 2, 50, seed=rep + 1, missing=0.2)
        q[q >= 50] = -1
        p.copy_(q)
        g.replay()
        torch.cuda.synchronize()
        _experts.check_combine_grad(dh, dw, dy, h, p, w, torch.zeros_like(h), "replay %d" % rep)
        dh.fill_(9.0)
        assert torch.equal(dg.combine_rows_grad(dy, h, p, w)[1], dw)
