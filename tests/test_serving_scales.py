"""The softmax scale of the attention calls: what is refused, and scales at the ends of what is
taken."""

import pytest
import torch

from tests import serving_reference as ref
from tests.test_gpu_serving import cross as run_cross
from tests.test_gpu_serving import decode as run_decode
from tests.test_gpu_serving import states
from tests.test_serving_refusals import EINVAL, cross, decode


@pytest.mark.parametrize("call", [decode, cross])
@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scales_beyond_the_exponents_range_are_refused(call, scale):
    assert call(scale=scale) == EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-30, 1.0, 30.0, 1000.0])
def test_scales_from_the_smallest_to_large_ones(scale, dtype):
    # powers of two in few elements: scores are exact, so large scales do not magnify rounding.
    # (The last tokens' -inf: a reference far from the scores must not matter at any scale.)
    n, g = 300, 4
    cache, kv = states([n], 1, dtype, 1)
    r = torch.Generator().manual_seed(2)
    k = torch.zeros((n, 1, 128))
    k[:, 0, 0] = torch.randint(-3, 4, (n,), generator=r).float()
    k[n - 140:n - 2, 0, 3] = -float("inf")
    k = k.to(dtype).cuda()
    v = kv[0][1]
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = torch.zeros((50, g, 128))
    q[..., 0] = torch.randint(-2, 3, (50, g), generator=r).float()
    q[..., 3] = 1.0
    q = q.to(dtype).cuda()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[n - 140:n - 2] = False
    s = float(torch.tensor(scale, dtype=torch.float32))
    want = ref.attention(q, k[keep], v[keep], s)
    ref.assert_close(run_cross(cache, 1, q, [50], [n], scale=scale), *want)
    ref.assert_close(run_decode(cache, 1, q[:1], [n], scale=scale), want[0][:1], want[1][:1])
