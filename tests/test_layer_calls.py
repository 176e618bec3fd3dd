"""The Python entry points of the layer products: what they hand to the C ABI,
and what they refuse.  On the CPU the device checks and the launch are replaced
(nothing runs); the GPU tests make the same calls in earnest."""
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
