"""The binding of the calls around the cache: what it refuses before the library is called."""

import pytest
import torch

from bit_quantization_head_b200 import kvtc


class HostCache:
    """A cache whose pool is on the host (RawCache itself refuses one)."""

    def __init__(self):
        self.pool = torch.zeros((1, 1, 1, 2, 128, 128), dtype=torch.bfloat16)
        self.desc = kvtc.RawCacheDesc(None, 1, 1, 1, kvtc.KVTC_BF16, None, 2, 1, None)
        self._address = kvtc.C.addressof(self.desc)


def host_calls():
    i, x = torch.zeros(4, dtype=torch.int32), torch.zeros((2, 3, 128), dtype=torch.bfloat16)
    c = HostCache()
    return [lambda: kvtc.kvtc_step_tables(i, i, i, i[:2], i.view(1, 4), i, i, i.long(), i, i[:2], i),
            lambda: kvtc.kvtc_rope(kvtc.rope_desc([64]), x, None, i[:2], x, None),
            lambda: kvtc.kvtc_rope(kvtc.rope_desc([64]), None, x, i[:2], None, x),
            lambda: kvtc.kvtc_raw_append(c, 0, x, x, i.long()),
            lambda: kvtc.kvtc_raw_decode_attention(c, 0, x, i[:2], 10, x, i),
            lambda: kvtc.kvtc_raw_cross_attention(c, 0, x, i[:3], i[:2], 10, x, i)]


@pytest.mark.parametrize("n", range(6))
def test_host_tensors_are_refused(n):
    with pytest.raises(ValueError, match="current CUDA device"):
        host_calls()[n]()


def test_what_is_no_tensor_is_refused():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="must be a tensor"):
        kvtc.kvtc_step_tables([0, 1], i, i, i[:2], i.view(1, 4), i, i, i.long(), i, i[:2], i)
    with pytest.raises(TypeError, match="must be a tensor"):
        kvtc.kvtc_rope(kvtc.rope_desc([64]), 3, None, i, i, None)
    with pytest.raises(ValueError, match="q or k"):
        kvtc.kvtc_rope(kvtc.rope_desc([64]), None, None, i, None, None)
    with pytest.raises(TypeError, match="unsupported dtype"):
        kvtc.kvtc_rope(kvtc.rope_desc([64]), torch.zeros((2, 3, 128), dtype=torch.float64), None, i, i, None)


# ------------------------------------------------------------------ buffers that overlap
A = 1 << 30          # stands for aligned device addresses far apart; never dereferenced


def raw_cache():
    return kvtc.RawCacheDesc(8 * A, 2, 64, 2, kvtc.KVTC_BF16, 9 * A, 3, 8, None)


def test_attention_refuses_outputs_and_workspaces_in_the_pool():
    L, c = kvtc.lib(), kvtc.C.byref(raw_cache())
    pool = 8 * A + 4096
    for q, out, ws in ((A, pool, 3 * A), (A, 2 * A, pool), (A, 3 * A + 4096, 3 * A), (3 * A + 256, 2 * A, 3 * A)):
        assert L.kvtc_raw_decode_attention(c, 0, q, 8, 4 * A, 1000, 0.0, out, ws, 1 << 29, None) == 1
        assert L.kvtc_raw_cross_attention(c, 0, q, 8, 5 * A, 100, 4 * A, 1000, 0.0, out, ws, 1 << 29, None) == 1


def test_append_refuses_rows_in_the_pool():
    L, c, pool = kvtc.lib(), kvtc.C.byref(raw_cache()), 8 * A + 8192
    d = kvtc.C.byref(kvtc.rope_desc([64]))
    for k, v, q, out in ((pool, A, 2 * A, 3 * A), (A, pool, 2 * A, 3 * A), (A, 4 * A, pool, 3 * A), (A, 4 * A, 2 * A, pool)):
        assert L.kvtc_raw_append(c, 0, k, 256, v, 256, 5 * A, 8, d, 6 * A, q, 512, 4, out, None) == 1
