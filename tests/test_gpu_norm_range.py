"""GPU tests of the norms of fp32 rows so small that their mean square is a subnormal float."""
import pytest
import torch

import semi_structured_sparse_amd as nm
from tests import block_bounds as ref
from tests.test_gpu_block import generator, near, normal

pytestmark = pytest.mark.gpu


def subnormal_slack(y, x, kind):
    """What a mean square q on the subnormals' grid may add to a norm's slack: each of a row's n additions and
    the product with 1 / n are off by 2^-150, which is 2^-149 of q at most relative to it, and rsqrt halves it
    (first order; twice that covers the rest)."""
    x = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    return y.abs() * 2.0 ** -149 / x.square().mean(-1, keepdim=True)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("size", [1e-17, 1e-18, 1e-19, 1e-20, 4e-21])
@pytest.mark.parametrize("width", [64, 500, 4100, 20000])
def test_small_rows_without_eps(kind, size, width):
    gen = generator(width)
    x = normal(gen, 5, width, dtype=torch.float32) * size
    weight = normal(gen, width)
    y = nm.nm_norm(x, weight, kind=kind, eps=0.0)
    want, slack = ref.norm(x.double(), weight.double(), None, kind, 0.0, 0.0)
    near(y, want, slack + subnormal_slack(want, x.double(), kind) + ref.half_rounding(want), f"norm {kind} {width} of {size}")
    branch = torch.zeros(5, width, dtype=torch.float16, device=x.device)
    z, h = nm.nm_block_norm(x, branch, weight, kind=kind, eps=0.0)
    assert torch.equal(h, x) and torch.equal(z, y)
