"""What a caller may do with one of route()'s results and the others stay as they
were, on the GPU."""
import pytest

import dense_gemm_08_amd as dg
from tests import _experts
from tests.test_gpu_route import logits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0, 1, 16, 128, 129, 5000])
def test_each_result_has_memory_of_its_own(T):
    # keeping or saving one keeps that one alone: no other result, no workspace
    l = logits(T, 40, "bf16")
    r = dg.route(l, 3)
    torch.cuda.synchronize()
    _experts.check_route(r, l, 3, "results")
    for name, t in zip(r._fields, r):
        assert t.is_contiguous() and t._base is None, name
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == 4 * t.numel(), name


class Gathered(torch.autograd.Function):
    """Rows gathered by token; the gradient adds them up by place."""

    @staticmethod
    def forward(ctx, x, tokens, places):
        ctx.save_for_backward(places)
        return x.index_select(0, tokens.clamp(min=0))

    @staticmethod
    def backward(ctx, g):
        return dg.combine_rows(g.contiguous(), ctx.saved_tensors[0]), None, None


@pytest.mark.parametrize("T", [30, 200])
def test_a_result_changed_in_place_leaves_what_autograd_saved(T):
    l = logits(T, 16, "f32")
    l[T - 4:] = -float("inf")                   # padding: rows of no token behind the others
    r = dg.route(l, 2)
    x = torch.randn((T, 24), device="cuda").bfloat16().requires_grad_()
    y = Gathered.apply(x, r.tokens, r.places)
    for t in (r.tokens, r.ends, r.experts):
        t.clamp_(min=0)
    y.sum().backward()
    want = torch.full_like(x, 2.0)
    want[T - 4:] = 0.0
    assert torch.equal(x.grad, want)


def test_too_many_choices_are_refused_before_memory_is_taken():
    # 2^25 tokens of 64 choices, by a view: their results would be 32 GB
    l = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda").expand(1 << 25, 64)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for k in (64, 65):
        with pytest.raises(dg.DenseGemmError) as err:
            dg.route(l, k)
        assert err.value.status == dg.Status.TOO_LARGE
    assert torch.cuda.max_memory_allocated() == before
