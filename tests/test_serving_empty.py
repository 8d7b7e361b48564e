"""Steps without tokens: empty tensors have null pointers, and every call takes them."""

import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests.test_serving_refusals import append, cross, desc, rope


def test_calls_without_tokens_take_null_rows():
    d = kvtc.C.byref(desc())
    none = dict(k=None, v=None, slots=None)
    assert append(n=0, d=d, **none, pos=None, q=None, qo=None) == 0
    assert append(n=0, d=d, **none, pos=None, q=None, qs=0, qh=0, qo=None) == 0
    assert append(n=0, d=None, **none, pos=None, q=None, qs=0, qh=0, qo=None) == 0
    assert rope(n=0, q=None, k=None, pos=None, qo=None, ko=None) == 0
    assert cross(n=0, q=None, out=None) == 0


@pytest.mark.gpu
def test_the_binding_takes_empty_tensors():
    cache = kvtc.RawCache(1, 2, 3, torch.zeros((1, 3), dtype=torch.int32))
    q, k = (torch.empty((0, h, 128), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    slots, pos = (torch.empty(0, dtype=t, device="cuda") for t in (torch.int64, torch.int32))
    r = kvtc.rope_desc([64])
    kvtc.kvtc_raw_append(cache, 0, k, k, slots)
    kvtc.kvtc_raw_append(cache, 0, k, k, slots, rope=r, positions=pos)
    kvtc.kvtc_raw_append(cache, 0, k, k, slots, rope=r, positions=pos, q=q, q_out=torch.empty_like(q))
    kvtc.kvtc_rope(r, q, k, pos, torch.empty_like(q), torch.empty_like(k))
    lens, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(1, 0, 4, 2, 10), dtype=torch.uint8, device="cuda")
    kvtc.kvtc_raw_cross_attention(cache, 0, q, cu, lens, 10, torch.empty_like(q), ws)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    state, ring = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    kvtc.kvtc_step_tables(lens, one, ring, state, cache.block_table, lens, cu, slots, pos, state,
                          torch.zeros(4, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert not cache.pool.any() and cache.status.item() == 0 and state.tolist() == [0, 3]
