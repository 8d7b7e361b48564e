"""The longest sequence that a block table can describe, 2^31 - 128 tokens: one page named again
and again, and another one at the very end."""

import math

import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests.test_gpu_serving import cross, decode

pytestmark = pytest.mark.gpu
P, D = 128, 128


@pytest.mark.parametrize("call", ["decode", "cross"])
@pytest.mark.parametrize("short", [0, 70])
def test_the_longest_sequence_of_a_block_table(call, short):
    # Every key scores 0 but the last, whose weight of e^24 outweighs the 2^31 others.  Sums of a
    # block's run: 113000 tiles or steps at most, added one by one (2^-24 each); the cross
    # kernel's weights of 1 enter the sum as 1 +- 2^-13.7.
    max_pages = (1 << 24) - 1
    n = max_pages * P - short
    table = torch.zeros((1, max_pages), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    cache = kvtc.RawCache(1, 1, 2, table)
    v = torch.randint(-1, 2, (P, D), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    cache.pool[0, 0, 0, 1] = v
    last = (n - 1) % P
    hot = torch.randint(-1, 2, (D,), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    cache.pool[0, 1, 0, 0, last, 0] = 24.0
    cache.pool[0, 1, 0, 1, last] = hot
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out = decode(cache, 0, q, [n], scale=1.0) if call == "decode" else cross(cache, 0, q, [1], [n], scale=1.0)
    w = math.exp(24.0)
    want = (v.double().sum(0) * (max_pages - 1) + hot.double() * w) / (n - 1 + w)
    assert cache.status.item() == 0
    tol = 113000 * 2.0 ** -24 + 2.0 ** -13.7 + 2.0 ** -8
    assert ((out[0, 0].double() - want).abs() <= tol * (want.abs() + 0.1)).all()
