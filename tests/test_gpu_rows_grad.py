"""What combine_rows_grad leaves where no place leads, and its results one by one, on
the GPU."""
import pytest

import dense_gemm_08_amd as dg
from tests import _experts, _layer
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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,N,k", [(1, 1, 1), (3, 7, 1), (33, 129, 5), (130, 1024, 8), (4, 4097, 3), (2, 16400, 9),
                                   (9000, 40, 3)])
def test_each_result_alone(T, N, k, dtype):
    # every number of lanes a row; the same bits as both together
    R = T * k + 3
    h, dy = values(R, N, dtype), values(T, N, dtype, seed=1)
    p, w = choices(T, k, R, missing=0.2)
    print("combine_grad alone", T, N, k, dtype, flush=True)
    for ww in (w, None):
        before = torch.full((R, N), 3.0, dtype=h.dtype, device="cuda")
        dh, dw = dg.combine_rows_grad(dy, h, p, ww, dh=before.clone())
        nan = torch.full_like(h, float("nan"))  # (h is not read)
        a, none = dg.combine_rows_grad(dy, nan, p, ww, dh=before.clone(), only="dh")
        assert none is None and torch.equal(a, dh)
        a, none = dg.combine_rows_grad(dy, nan, p, ww, only="dh")
        _experts.check_combine_grad(a, dw, dy, h, p, ww, torch.zeros_like(h), "dh alone")
        none, b = dg.combine_rows_grad(dy, h, p, ww, only="dweights")
        assert none is None and torch.equal(b, dw)


def test_alone_where_there_is_little():
    h, dy = values(6, 24, "bf16"), values(3, 24, "bf16", seed=1)
    p = torch.tensor([[0, 5], [1, 3], [2, 4]], dtype=torch.int32, device="cuda")
    # rows of no columns have a gradient of the rows, as they have a sum
    assert dg.combine_rows(h[:, :0], p).shape == (3, 0)
    dh, none = dg.combine_rows_grad(dy[:, :0], h[:, :0], p, only="dh")
    assert dh.shape == (6, 0) and none is None
    # no rows at all, no tokens
    dh, none = dg.combine_rows_grad(dy, h[:0], p, only="dh")
    assert dh.shape == (0, 24) and none is None
    none, dw = dg.combine_rows_grad(dy, h[:0], p, only="dweights")
    assert (dw == 0).all()
    dh, none = dg.combine_rows_grad(dy[:0], h, p[:0], only="dh")
    assert (dh == 0).all() and dh.shape == h.shape
    none, dw = dg.combine_rows_grad(dy[:0], h, p[:0], only="dweights")
    assert dw.shape == (0, 2)
    with pytest.raises(ValueError):
        dg.combine_rows_grad(dy, h, p, only="weights")
    with pytest.raises(ValueError):
        dg.combine_rows_grad(dy, h, p, dh=h, only="dweights")
    with pytest.raises(dg.DenseGemmError):
        dg.combine_rows_grad(dy[:, :0], h[:, :0], p, only="dweights")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,N,k,R", [(4, 24, 2, 3), (40, 130, 3, 17), (50, 1024, 1, 9), (9, 40, 6, 1)])
def test_rows_named_more_than_once_get_their_gradient_by_a_combination(T, N, k, R, dtype):
    # what combine_rows' docstring says to do where places repeat
    g = torch.Generator().manual_seed(T + N)
    p = torch.randint(-1, R, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand((T, k), generator=g)
    h, dy = values(R, N, dtype), values(T, N, dtype, seed=1)
    of = [[(t, j) for t in range(T) for j in range(k) if p[t, j] == r] for r in range(R)]
    m = max(len(x) for x in of)
    assert 1 < m <= 64
    places = torch.full((R, m), -1, dtype=torch.int32)
    weights = torch.zeros((R, m))
    for r, x in enumerate(of):
        for i, (t, j) in enumerate(x):
            places[r, i], weights[r, i] = t, w[t, j]
    p, w, places, weights = p.cuda(), w.cuda(), places.cuda(), weights.cuda()
    dh = dg.combine_rows(dy, places, weights)
    _experts.check_combine(dh, dy, places, weights, None, "sums of the choices")
    # the same sums from the definition
    rows, there = _experts.rows64(h, p)
    hd = h.double().requires_grad_()
    y = (torch.where(there[:, :, None], hd[p.long().clamp(min=0)], torch.zeros_like(rows)) * w.double()[:, :, None]).sum(1)
    y.backward(dy.double())
    terms, _ = _experts.rows64(dy, places)
    S = (terms * weights.double()[:, :, None]).abs().sum(1)
    off = (dh.double() - hd.grad).abs()
    assert (off <= m * 2.0 ** -24 * S * 1.02 + _layer.rounding(hd.grad, h.dtype) * 1.01).all()
    # the weights' gradient does not mind
    _, dw = dg.combine_rows_grad(dy, h, p, w, only="dweights")
    s, S = (rows * dy.double()[:, None, :]).sum(2), (rows * dy.double()[:, None, :]).abs().sum(2)
    _layer.assert_close(dw, s, S * (N + 16) * 2.0 ** -24 * 1.01 + 2.0 ** -24 * s.abs(), "dweights")
