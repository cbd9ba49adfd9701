"""The operators between the adapted linears at the ends of their ranges: tails
of the activations, far positions, long sums, and calls whose CTAs leave while
the other one of a pair has just finished.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def am(cuda_device):
    from adapter_merge_b200 import build
    build.build()
    import adapter_merge_b200
    adapter_merge_b200.lib()
    return adapter_merge_b200


def rnd(*shape, seed=0, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("T", [513, 600, 640, 1025])
def test_pairs_whose_second_cta_stores_nothing_last(am, T):
    """1 to 128 tokens in the last tile: the pair's second CTA gives its
    accumulator back and is done at once.  Many calls back to back, so that each
    finds shared memory that the last one has just left."""
    assert 1 <= T % 256 <= 128
    x, W, U = rnd(T, 128), rnd(1024, 128, seed=1, std=0.05), rnd(1024, 128, seed=2, std=0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for f in (lambda: am.project(x, W, status=status), lambda: am.project(x, W, out_dtype=F32, status=status),
              lambda: am.gated_project(x, W, U, status=status)):
        first = f()
        assert all(torch.equal(first, y) for y in [f() for _ in range(40)])
    assert int(status) == 0
