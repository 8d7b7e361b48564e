"""The coded cache's entry points of the library take fp32 and bf16: fp16, which the calls around
the cache know, is refused by each of them (it must not be read as one of the others)."""

import numpy as np
import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests import gpu_helpers as gh

pytestmark = pytest.mark.gpu
EINVAL = 1


def test_every_coded_entry_point_refuses_f16():
    L, H, G = kvtc.lib(), 2, 2
    plan = gh.random_plan(1, H, G, [((64, 4), (64, 4))] * H, np.random.default_rng(1))
    cache = kvtc.Cache(plan, 2, torch.arange(2, dtype=torch.int32).view(1, 2))
    c, h = kvtc.C.byref(cache.desc), plan.handle
    x = torch.zeros((4, H * G, 128), dtype=torch.float32, device="cuda")
    i32 = torch.tensor([0, 4], dtype=torch.int32, device="cuda")  # offsets; a length of 0
    slots = torch.arange(4, device="cuda")
    ws = torch.zeros(kvtc.kvtc_decode_workspace_bytes(plan, 1, 4), dtype=torch.uint8, device="cuda")
    out = torch.full((1, H * G, 128), 7.0, device="cuda")
    p, n = (lambda t: t.data_ptr()), ws.numel()
    f16, f32 = kvtc.KVTC_F16, kvtc.KVTC_F32
    calls = {
        "append": lambda t: L.kvtc_encode_append(h, c, 0, p(x), p(x), t, p(i32), p(i32), 4, None),
        "append_slots": lambda t: L.kvtc_encode_append_slots(h, c, 0, p(x), p(x), t, p(slots), 4, None),
        "latent": lambda t: L.kvtc_debug_encode_latent(h, 0, 0, 0, p(x), t, 1, p(x) + 1024, None),
        "decode q": lambda t: L.kvtc_decode_attention(h, c, 0, p(x), t, p(i32), 4, 0.0, p(out), f32, p(ws), n, None),
        "decode out": lambda t: L.kvtc_decode_attention(h, c, 0, p(x), f32, p(i32), 4, 0.0, p(out), t, p(ws), n, None),
        "noalloc q": lambda t: L.kvtc_decode_attention_noalloc(h, c, 0, p(x), t, p(i32), 4, 0.0, p(out), f32, None),
        "noalloc out": lambda t: L.kvtc_decode_attention_noalloc(h, c, 0, p(x), f32, p(i32), 4, 0.0, p(out), t, None),
        "rope q": lambda t: L.kvtc_decode_attention_rope(h, c, 0, p(x), t, p(i32), 4, 0.0, 0.0, p(out), f32, p(ws), n, None),
        "rope out": lambda t: L.kvtc_decode_attention_rope(h, c, 0, p(x), f32, p(i32), 4, 0.0, 0.0, p(out), t, p(ws), n, None),
    }
    for name, call in calls.items():
        for bad in (f16, 3, -1):
            assert call(bad) == EINVAL, name
            assert b"dtype must be F32 or BF16" in L.kvtc_last_error(), name
    torch.cuda.synchronize()
    assert not cache.pool.any() and (out == 7.0).all()
    for name, call in calls.items():
        assert call(f32) == 0, name                     # the same calls but for the type
    torch.cuda.synchronize()
    assert cache.status.item() == 0
