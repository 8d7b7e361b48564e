"""Attention rows depend on their own query, keys and values alone: the same bits again, after
other calls have used the chip, from another place in memory, and beside other rows."""

import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests.test_gpu_serving import cross, decode, i32, states

pytestmark = pytest.mark.gpu
D = 128
TYPES = [torch.bfloat16, torch.float16]


def rand_q(n, hq, dtype, seed, scale=1.0):
    return (torch.randn((n, hq, D), generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hk,lens,q_lens", [(3, 1, [4000], [100]), (8, 2, [2500, 900], [40, 33]), (5, 1, [700], [2]),
                                               (100, 1, [3000], [3])])
def test_cross_rows_do_not_depend_on_rows_behind_them(hq, hk, lens, q_lens, dtype):
    # rows behind the last sequence share its tiles: whatever they hold, its rows stay the same
    cache, _ = states(lens, hk, dtype, 1)
    n, cu = sum(q_lens), [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    q = rand_q(n + 130, hq, dtype, 2, 3.0)
    first = None
    for scale in (0.0, 1.0, 30.0, float("nan"), float("inf")):
        q[n:] = rand_q(130, hq, dtype, 3, 4.0) * scale
        out = cross(cache, 1, q, None, lens, cu=cu)
        assert torch.isfinite(out[:n]).all() and (out[n:] == 123.0).all()
        first = out if first is None else first
        assert torch.equal(out[:n], first[:n])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("g", [3, 5, 7, 100])
def test_cross_rows_do_not_depend_on_what_ran_before(g, dtype):
    # tiles whose tokens' heads do not fill 128 rows leave some that no load writes
    cache, _ = states([5000], 1, dtype, 4)
    q = rand_q(150, g, dtype, 5, 3.0)
    first = cross(cache, 1, q, [150], [5000])
    for scale in (0.0, 1.0, 30.0):
        cross(cache, 1, rand_q(40000, 1, dtype, 6, 4.0) * scale, [40000], [5000])   # fills every tile's rows
        assert torch.equal(cross(cache, 1, q, [150], [5000]), first)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,q_lens,hq,hk", [([1000, 0, 517], [4, 1, 17], 32, 8), ([20000], [300], 28, 4),
                                               ([9000] * 4, [500, 3, 70, 1], 20, 20), ([50000], [2], 8, 1)])
def test_the_same_bits_every_time_and_everywhere(lens, q_lens, hq, hk, dtype):
    n, copies = sum(q_lens), []
    for _ in range(2):                                  # the same inputs in two places
        cache, _ = states(lens, hk, dtype, 7)
        copies.append((cache, rand_q(len(lens), hq, dtype, 8), rand_q(n, hq, dtype, 9)))
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        cache, qd, qx = copies[i & 1]
        if i % 3 == 0:
            big.fill_(i)                                # cold pages
        got = decode(cache, 1, qd, lens), cross(cache, 1, qx, q_lens, lens)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_decode_joins_groups_of_parts_the_same_way_every_time():
    # more than 48 parts of 5 to 8 heads: groups of parts are joined into the place of their first
    for hq in (5, 8):
        cache, _ = states([60000], 1, torch.bfloat16, 10)
        q, sl = rand_q(1, hq, torch.bfloat16, 11), i32([60000])
        ws = torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(1, hq, 1, 60000), dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(q) for _ in range(200)]
        for out in outs:
            kvtc.kvtc_raw_decode_attention(cache, 1, q, sl, 60000, out, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(out, outs[0]) for out in outs)
