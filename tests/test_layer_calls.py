"""The Python entry points of the layer products: what they hand to the C ABI,
and what they refuse.  On the CPU the device checks and the launch are replaced
(nothing runs); the GPU tests make the same calls in earnest."""
import ctypes
import importlib.util
import sys

import pytest
import torch

import dense_gemm_08_amd as dg
from dense_gemm_08_amd import binding

S = binding.Status


@pytest.fixture
def handed(monkeypatch):
    """The list of (name, arguments) that calls on host tensors hand to the
    launch."""
    calls = []
    monkeypatch.setattr(binding, "_check_first", lambda A: (binding._FMTS[A.dtype], A.dtype, -1))
    monkeypatch.setattr(binding, "_launch", lambda name, args, *rest: calls.append((name, args)))
    return calls


def test_first_calls_of_two_threads(monkeypatch):
    # a second thread's call may come in wherever the first one looks at torch:
    # the table of types is then whole, or still to be made
    spec = importlib.util.spec_from_file_location("fresh_binding", binding.__file__)
    fresh = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fresh)
    seen = []

    class Watched:
        def __getattr__(self, name):
            seen.append(set(fresh._FMTS or ()))
            return getattr(torch, name)

    monkeypatch.setitem(sys.modules, "torch", Watched())
    fresh._torch()
    whole = {torch.float16, torch.bfloat16}
    assert seen and all(types in (set(), whole) for types in seen)
    assert set(fresh._FMTS) == whole


def gradient_calls(device):
    A = torch.ones((4, 8), dtype=torch.bfloat16, device=device)
    ends = torch.tensor([4], dtype=torch.int32, device=device)
    nt, nn = A.new_ones((6, 8)), A.new_ones((8, 6))
    z = A.new_ones((4, 6))
    return z, [lambda z, act: dg.gemm_nt_dact(A, nt, z, act),
               lambda z, act: dg.gemm_nn_dact(A, nn, z, act),
               lambda z, act: dg.gemm_nt_grouped_dact(A, nt[None], ends, z, act),
               lambda z, act: dg.gemm_nn_grouped_dact(A, nn[None], ends, z, act)]


def test_gradient_calls_always_carry_their_form(handed):
    z, calls = gradient_calls("cpu")
    for call in calls:
        for zz, act in ((None, "none"), (z, "none"), (None, "silu"), (z, "silu")):
            call(zz, act)
            name, args = handed[-1]
            assert name == "dense_gemm_layer"
            epi = args[-2]
            assert epi is not None and epi.grad == 1 and epi.act == binding.ACTS[act]
            assert bool(epi.preact) == (zz is not None)


def test_no_groups_need_no_operands():
    lib = binding.load_library()
    none = binding.Groups(None, 0, 0)
    size = ctypes.c_size_t(7)
    for op in range(4):
        for A, D in ((None, None), (256, 256)):
            assert lib.dense_gemm_layer(op, 5, 6, 8, A, 8, None, 8, D, 6, None, none, None, 0, None) == S.OK
        assert lib.dense_gemm_layer_workspace_size(op, 5, 6, 8, 256, 8, None, 8, none, 256,
                                                   ctypes.byref(size)) == S.OK and size.value == 0
        # what is wrong whatever the groups hold stays refused
        assert lib.dense_gemm_layer(op, -5, 6, 8, None, 8, None, 8, None, 6, None, none, None, 0,
                                    None) == S.INVALID_DIM
        assert lib.dense_gemm_layer(op, 5, 6, 8, None, 8, None, 8, None, 6, binding.Epilogue(act=9), none,
                                    None, 0, None) == S.BAD_ARG
        assert lib.dense_gemm_layer(op, 5, 6, 8, None, 8, None, 8, None, 6, None,
                                    binding.Groups(None, 0, -1), None, 0, None) == S.BAD_ARG
        one = binding.Groups(256, 1, 0)
        assert lib.dense_gemm_layer(op, 5, 6, 8, 256, 8, None, 8, 256, 6, None, one, None, 0,
                                    None) == S.NULL_PTR
    assert lib.dense_gemm_tn(1, 5, 6, 8, None, 5, None, 6, None, 6, None, none, None, 0, None) == S.OK


@pytest.mark.gpu
def test_empty_stacks_of_matrices():
    A = torch.ones((5, 8), dtype=torch.bfloat16, device="cuda")
    ends = torch.empty((0,), dtype=torch.int32, device="cuda")
    D = torch.full((5, 6), 77.0, dtype=torch.bfloat16, device="cuda")
    z = torch.ones_like(D)
    nt, nn = A.new_empty((0, 6, 8)), A.new_empty((0, 8, 6))
    dg.gemm_nt_grouped(A, nt, ends, bias=A.new_empty((0, 6)), act="gelu", residual=z, D=D)
    dg.gemm_nn_grouped(A, nn, ends, D=D)
    dg.gemm_nt_grouped_dact(A, nt, ends, z, "relu", D=D)
    dg.gemm_nn_grouped_dact(A, nn, ends, z, "relu", D=D)
    assert bool((D == 77.0).all())
    W, c = dg.gemm_tn_grouped(A, z, ends, colsum=True)
    assert W.shape == (0, 8, 6) and c.shape == (0, 8)


@pytest.mark.gpu
def test_gradient_calls_without_an_activation_or_z_are_refused():
    z, calls = gradient_calls("cuda")
    for call in calls:
        for zz, act, status in ((None, "none", S.BAD_ARG), (z, "none", S.BAD_ARG),
                                (None, "silu", S.NULL_PTR)):
            with pytest.raises(dg.DenseGemmError) as e:
                call(zz, act)
            assert e.value.status == status
        call(z, "silu")
    torch.cuda.synchronize()


def grouped_bytes(op, M, N, K, count, stride):
    size = ctypes.c_size_t()
    ld = K if op in (0, 2) else N
    assert binding.load_library().dense_gemm_layer_workspace_size(
        op, M, N, K, 256, K, 256, ld, binding.Groups(256, count, stride), 256, ctypes.byref(size)) == S.OK
    return size.value


def test_a_matrix_that_all_groups_share_is_copied_once():
    rounded = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for op, rows, cols in ((0, 64, 129), (2, 64, 129), (1, 130, 65), (3, 130, 65)):
        N, K = (rows, cols) if op in (0, 2) else (cols, rows)
        a = rounded(500 * 136 * 2) if K % 2 else 0
        one = rows * ((cols + 7) // 8 * 8) * 2
        assert grouped_bytes(op, 500, N, K, 7, 0) == a + rounded(one)
        assert grouped_bytes(op, 500, N, K, 7, rows * cols) == a + rounded(7 * one)
        assert grouped_bytes(op, 500, N, K, 1, rows * cols) == a + rounded(one)
    # 64 groups of 4096 x 4097: 34 MB, not 2.1 GB
    assert grouped_bytes(2, 512, 4096, 4097, 64, 0) == 4096 * 4104 * 2 + 512 * 4104 * 2


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["nt", "nn"])
@pytest.mark.parametrize("sizes", [[30, 0, 200, 5], [3, 0, 1, 2], [700, 900, 0, 800]])
def test_a_shared_copied_matrix_gives_what_a_stack_of_it_gives(sizes, layout):
    gen = torch.Generator(device="cuda").manual_seed(len(sizes) + sizes[0])
    M, N, K, G = sum(sizes), 91, 105, len(sizes)
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    A = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    W = torch.randn((N, K) if layout == "nt" else (K, N), generator=gen, device="cuda").bfloat16()
    f = dg.gemm_nt_grouped if layout == "nt" else dg.gemm_nn_grouped
    # (a workspace of the size asked for and no more, the bytes behind it kept)
    need = grouped_bytes(2 if layout == "nt" else 1, M, N, K, G, 0)
    ws = torch.full((need + 256,), 55, dtype=torch.uint8, device="cuda")
    D = f(A, W.expand(G, *W.shape), ends, workspace=ws[:need])
    assert torch.equal(D, f(A, torch.stack([W] * G), ends))
    assert bool((ws[need:] == 55).all())
