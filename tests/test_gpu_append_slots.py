"""Coded rows of a serving step: rows that belong to no sequence leave every sequence's codes as
they are."""

import numpy as np
import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests import gpu_helpers as gh

pytestmark = pytest.mark.gpu
P, D, H = 128, 128, 2


def plan_of(seed, k_only=False):
    v = (128, kvtc.RAW_BITS) if k_only else (24, 5)
    return gh.random_plan(2, H, 2, [((64, 4), v), ((32, 2), v)] * 2, np.random.default_rng(seed))


def rows(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((n, H, D), generator=g).to(dtype).cuda() for _ in range(2)]


@pytest.mark.parametrize("n_seq", [127, 128, 129, 300])
def test_append_rows_behind_the_last_sequence_are_reported_and_not_written(n_seq):
    # 5 rows more than cu_seqlens covers; the last sequence's table still names pages of others
    plan = plan_of(1)
    table = torch.arange(n_seq * 2, dtype=torch.int32).view(n_seq, 2)
    table[-1, 1] = table[0, 0]
    cache, want = kvtc.Cache(plan, 2 * n_seq, table), kvtc.Cache(plan, 2 * n_seq, table)
    k, v = rows(n_seq + 5, torch.bfloat16, 2)
    start = torch.full((n_seq,), 125, dtype=torch.int32, device="cuda")
    cu = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda")
    kvtc.kvtc_encode_append(plan, want, 1, k[:n_seq], v[:n_seq], cu, start)
    kvtc.kvtc_encode_append(plan, cache, 1, k, v, cu, start)
    torch.cuda.synchronize()
    assert want.status.item() == 0 and want.pool.any()
    assert torch.equal(cache.pool, want.pool)
    assert cache.status.item() == kvtc.STATUS_BAD_POS
    # rows before the first sequence's are outside too
    cache.pool.copy_(want.pool)
    cache.status.zero_()
    kvtc.kvtc_encode_append(plan, cache, 1, k[:n_seq], v[:n_seq], cu + n_seq, start)
    torch.cuda.synchronize()
    assert torch.equal(cache.pool, want.pool) and cache.status.item() == kvtc.STATUS_BAD_POS
