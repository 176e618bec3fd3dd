"""Row groups by the thousand: their tiles are found by walking the ends of the
groups past those that the kernels hold in registers."""
import pytest
import torch

import dense_gemm_08_amd as dg

pytestmark = pytest.mark.gpu


def sample(G, seed, layout, N=40, K=24):
    """G groups of 0 to 3 rows and a few long ones, integers small enough for
    exact sums; the groups' ends, and each row's group."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    sizes = torch.randint(0, 4, (G,), generator=gen, device="cuda")
    sizes[torch.randint(0, G, (5,), generator=gen, device="cuda")] = 300
    ends = sizes.cumsum(0).to(torch.int32)
    rows = int(ends[-1]) + 9
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), sizes)

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device="cuda").bfloat16()

    return ints(rows, K), ints(*((G, N, K) if layout == "nt" else (G, K, N))), ends, group


@pytest.mark.parametrize("layout", ["nt", "nn"])
@pytest.mark.parametrize("G", [257, 1000, 1 << 13, (1 << 15) + 77])
def test_every_row_meets_its_groups_matrix(G, layout):
    A, B, ends, group = sample(G, G, layout)
    f = dg.gemm_nt_grouped if layout == "nt" else dg.gemm_nn_grouped
    D = torch.full((A.shape[0], 40), 77.0, dtype=A.dtype, device="cuda")
    f(A, B, ends, D=D)
    n = group.numel()
    want = torch.zeros((n, 40), dtype=torch.float32, device="cuda")
    for k in range(A.shape[1]):  # (sums of at most 24 x 9: exact in 32 bits and in BF16)
        b = B[:, :, k] if layout == "nt" else B[:, k, :]
        want += A[:n, k, None].float() * b.float()[group]
    assert torch.equal(D[:n].float(), want)
    assert bool((D[n:] == 77.0).all())


@pytest.mark.parametrize("layout", ["nt", "nn"])
def test_a_few_rows_among_thousands_of_groups(layout):
    # the small-output kernel, which holds 64 groups
    G, N, K = 5000, 40, 24
    gen = torch.Generator(device="cuda").manual_seed(5)
    group = torch.randint(0, G, (19,), generator=gen, device="cuda").sort().values
    group[1] = group[0]
    ends = torch.bincount(group, minlength=G).cumsum(0).to(torch.int32)
    A = torch.randint(-3, 4, (19, K), generator=gen, device="cuda").bfloat16()
    B = torch.randint(-3, 4, (G, N, K), generator=gen, device="cuda").bfloat16()
    want = (A[:, None].float() * B[group].float()).sum(-1)
    if layout == "nt":
        D = dg.gemm_nt_grouped(A, B, ends)
    else:
        D = dg.gemm_nn_grouped(A, B.transpose(1, 2).contiguous(), ends)
    assert torch.equal(D.float(), want)


def test_the_ends_are_walked_once_and_not_for_each_tile():
    # 2^15 groups of one row: 512 chunks of 64 ends.  Two walks at some 2 us a
    # chunk are 2 ms (measured: 1.0); a walk from the start for each of a
    # workgroup's 64 tiles is 32 times as many chunks (measured at half as many
    # groups: 4.9 ms, growing with their square).
    G = 1 << 15
    A = torch.ones((G, 8), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((1, 8, 8), dtype=torch.bfloat16, device="cuda").expand(G, 8, 8)
    ends = torch.arange(1, G + 1, dtype=torch.int32, device="cuda")
    D = dg.gemm_nt_grouped(A, B, ends)
    assert bool((D == 8).all())
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        dg.gemm_nt_grouped(A, B, ends, D=D)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    print("us", [round(t * 1e3) for t in times])
    assert min(times) < 6.0
