"""Argument checks of the calls around the cache (no GPU: each fails before a launch)."""

import ctypes as C

import pytest
import torch

from bit_quantization_head_b200 import kvtc

A = 1 << 20          # stands for aligned device addresses far apart; never dereferenced
EINVAL, ECAPACITY = 1, 5


def addr(i):
    return 64 * A * (i + 1)


def tables(**change):
    args = dict(cached=addr(0), new=addr(1), n_seq=4, ring=addr(2), capacity=16, state=addr(3), table=addr(4),
                max_pages=8, seq=addr(5), cu=addr(6), slots=addr(7), pos=addr(8), rows=10, out=addr(9), ws=addr(10),
                status=None)
    args.update(change)
    return kvtc.lib().kvtc_step_tables(*args.values(), None)


@pytest.mark.parametrize("change", [
    dict(n_seq=0), dict(n_seq=-1), dict(max_pages=0), dict(max_pages=1 << 24), dict(capacity=0), dict(rows=-1),
    dict(cached=None), dict(new=None), dict(ring=None), dict(state=None), dict(table=None), dict(seq=None),
    dict(cu=None), dict(slots=None), dict(pos=None), dict(out=None), dict(ws=None), dict(slots=addr(7) + 4),
    dict(cached=addr(0) + 2), dict(seq=addr(0) + 4), dict(cu=addr(0)), dict(out=addr(3) + 4), dict(ring=addr(4)),
    dict(pos=addr(7) + 76), dict(status=addr(10)), dict(new=addr(0))])
def test_step_tables_refuses(change):
    assert tables(**change) == EINVAL


def desc(sections=(64,), interleaved=0, base=0.0, n_axes=None):
    s = list(sections) + [0] * (4 - len(sections))
    return kvtc.RopeDesc(len(sections) if n_axes is None else n_axes, (C.c_int * 4)(*s), interleaved, base)


def rope(d=None, **change):
    args = dict(q=addr(0), qs=512, qh=4, k=addr(1), ks=256, kh=2, dtype=kvtc.KVTC_BF16, pos=addr(2), n=8, inverse=0,
                qo=addr(3), ko=addr(4))
    args.update(change)
    return kvtc.lib().kvtc_rope(C.byref(d or desc()), *args.values(), None)


@pytest.mark.parametrize("d", [desc(n_axes=0), desc(n_axes=5), desc((63,)), desc((65,)), desc((32, 33)),
                               desc((-1, 65)), desc(base=1.0), desc(base=-2.0), desc(base=float("nan")),
                               desc(base=float("inf")), desc((16, 24, 20))])
def test_rope_refuses_descriptions(d):
    assert rope(d) == EINVAL


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(dtype=-1), dict(n=-1), dict(q=None), dict(k=None), dict(pos=None), dict(qo=None),
    dict(ko=None), dict(qs=511), dict(qs=516), dict(qs=504), dict(qh=0), dict(qh=1025, qs=1 << 18), dict(q=addr(0) + 2),
    dict(qo=addr(3) + 8), dict(qo=addr(0) + 1024), dict(qo=addr(0), qs=1024), dict(q=None, qh=0, k=None, kh=0),
    dict(ko=addr(3)), dict(qo=addr(1)), dict(ko=addr(0) + 4096)])
def test_rope_refuses(change):
    assert rope(**change) == EINVAL


def test_rope_of_no_tokens_is_a_no_op():
    assert rope(n=0) == 0


def cache(**change):
    args = dict(pool=addr(20), n_layers=2, n_pages=64, n_kv_heads=2, dtype=kvtc.KVTC_BF16, block_table=addr(21), n_seq=3,
                max_pages=8, status=None)
    args.update(change)
    return kvtc.RawCacheDesc(*args.values())


BAD_CACHES = [dict(pool=None), dict(pool=addr(20) + 64), dict(n_layers=0), dict(n_pages=0), dict(n_kv_heads=0),
              dict(n_kv_heads=1025), dict(dtype=kvtc.KVTC_F32), dict(dtype=7), dict(n_pages=1 << 22),
              dict(n_pages=1 << 63), dict(n_layers=1 << 30)]


def append(c=None, layer=1, d=None, **change):
    args = dict(k=addr(0), ks=256, v=addr(1), vs=256, slots=addr(2), n=8)
    more = dict(pos=addr(3), q=addr(4), qs=512, qh=4, qo=addr(5))
    for key, val in change.items():
        (args if key in args else more)[key] = val
    return kvtc.lib().kvtc_raw_append(C.byref(c or cache()), layer, *args.values(), d, *more.values(), None)


@pytest.mark.parametrize("change", BAD_CACHES)
def test_raw_append_refuses_caches(change):
    assert append(cache(**change), d=C.byref(desc())) == EINVAL


@pytest.mark.parametrize("change", [
    dict(layer=-1), dict(layer=2), dict(n=-1), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None),
    dict(qo=None), dict(q=None), dict(ks=255), dict(vs=252), dict(k=addr(0) + 8), dict(v=addr(1) + 2),
    dict(q=addr(4) + 4), dict(qo=addr(5) + 4), dict(qs=256), dict(qo=addr(4) + 512), dict(qo=addr(0)), dict(qo=addr(1))])
def test_raw_append_refuses(change):
    assert append(d=C.byref(desc()), **change) == EINVAL
    if "pos" not in change and "q" not in change:
        assert append(d=None, **change) == EINVAL  # q without a rope description


def test_raw_append_of_no_tokens_is_a_no_op():
    assert append(n=0, d=C.byref(desc())) == 0


def decode(c=None, layer=0, **change):
    args = dict(q=addr(0), hq=8, lens=addr(1), mx=1000, scale=0.0, out=addr(2), ws=addr(3), wb=1 << 40)
    args.update(change)
    return kvtc.lib().kvtc_raw_decode_attention(C.byref(c or cache()), layer, *args.values(), None)


def cross(c=None, layer=0, **change):
    args = dict(q=addr(0), hq=8, cu=addr(4), n=100, lens=addr(1), mx=1000, scale=0.0, out=addr(2), ws=addr(3),
                wb=1 << 40)
    args.update(change)
    return kvtc.lib().kvtc_raw_cross_attention(C.byref(c or cache()), layer, *args.values(), None)


@pytest.mark.parametrize("call", [decode, cross])
@pytest.mark.parametrize("change", BAD_CACHES + [dict(block_table=None), dict(n_seq=0), dict(max_pages=0),
                                                 dict(max_pages=1 << 24)])
def test_attention_refuses_caches(call, change):
    assert call(cache(**change)) == EINVAL


@pytest.mark.parametrize("call", [decode, cross])
@pytest.mark.parametrize("change", [
    dict(layer=-1), dict(layer=2), dict(q=None), dict(lens=None), dict(out=None), dict(ws=None), dict(hq=0), dict(hq=7),
    dict(hq=4096), dict(mx=-1), dict(mx=1025), dict(scale=float("nan")), dict(scale=-1.0), dict(scale=float("inf")),
    dict(q=addr(0) + 8), dict(out=addr(2) + 2), dict(ws=addr(3) + 4), dict(out=addr(0)), dict(out=addr(0) + 256)])
def test_attention_refuses(call, change):
    assert call(**change) == EINVAL


def test_attention_refuses_small_workspaces_and_row_counts():
    L = kvtc.lib()
    need = L.kvtc_raw_decode_workspace_bytes(3, 8, 2, 1000)
    assert need > 0 and decode(wb=need - 1) == ECAPACITY
    need = L.kvtc_raw_cross_workspace_bytes(3, 100, 8, 2, 1000)
    assert need > 0 and cross(wb=need - 1) == ECAPACITY
    assert cross(n=-1) == EINVAL and cross(cu=None) == EINVAL
    assert cross(n=0) == 0
    assert cross(cache(n_kv_heads=1), hq=129) == EINVAL      # more than 128 query heads per KV head
    for bad in [(0, 8, 2, 10), (1, 1, 2, 10), (1, 8, 0, 10), (1, 8, 2, -1)]:
        assert L.kvtc_raw_decode_workspace_bytes(*bad) == 0
    for bad in [(0, 5, 8, 2, 10), (1, -1, 8, 2, 10), (1, 5, 1, 2, 10), (1, 5, 8, 0, 10), (1, 5, 8, 2, -1)]:
        assert L.kvtc_raw_cross_workspace_bytes(*bad) == 0


def test_raw_cache_bytes():
    L = kvtc.lib()
    assert L.kvtc_raw_cache_bytes(2, 5, 3) == 2 * 5 * 3 * 2 * 128 * 128 * 2
    assert L.kvtc_raw_cache_bytes(0, 5, 3) == L.kvtc_raw_cache_bytes(2, 0, 3) == L.kvtc_raw_cache_bytes(2, 5, 0) == 0


def test_the_coded_cache_still_refuses_f16():
    # F16 belongs to the calls around the cache; the coded calls' dtype checks come first
    with pytest.raises(TypeError):
        kvtc._dtype_code(torch.zeros(1, dtype=torch.float16))


def test_binding_refuses_host_tensors_and_shapes():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvtc.kvtc_step_tables(i32, i32, i32, i32[:2], i32.view(1, 4), i32, i32, i32.long(), i32, i32[:2], i32)
    x = torch.zeros((2, 3, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kvtc.kvtc_rope(kvtc.rope_desc([64]), x, None, i32[:2], x, None)
    with pytest.raises(ValueError):
        kvtc.kvtc_rope(kvtc.rope_desc([64]), None, None, i32[:2], None, None)
    with pytest.raises(ValueError):
        kvtc.rope_desc([])
    with pytest.raises(ValueError):
        kvtc.rope_desc([16, 16, 16, 8, 8])
    with pytest.raises(ValueError):
        kvtc.RawCache(1, 1, 1, i32.view(1, 4), pool=torch.zeros((1, 1, 1, 2, 128, 128), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        kvtc.RawCache(1, 1, 1, i32.view(1, 4), dtype=torch.float32)
