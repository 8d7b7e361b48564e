"""Scores that are infinite: a key whose score is -inf has weight zero wherever it stands, rows
whose every score is -inf (and rows with a score of +inf) have no softmax and are NaN, and no
other row sees any of it."""

import pytest
import torch

from tests import serving_reference as ref
from tests.test_gpu_serving import cross, decode, states

pytestmark = pytest.mark.gpu
D = 128
TYPES = [torch.bfloat16, torch.float16]
INF = float("inf")

# tokens and those among them whose key scores -inf (in KV head 1)
CASES = [(17, [16]), (17, list(range(16))), (1, []), (2, [0]), (64, list(range(16, 32))), (200, list(range(64))),
         (300, list(range(128))), (300, list(range(256))), (300, [t for t in range(300) if t % 64 < 16]),
         (300, list(range(1, 300))), (300, list(range(299))), (700, list(range(512))), (1500, list(range(128, 1500, 2))),
         (9000, list(range(5000))), (9000, list(range(4000, 9000)))]


def queries(n, hq, dtype, seed):
    q = torch.randn((n, hq, D), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    q[..., 5] = q[..., 5].abs() + 0.5
    return q


def cache_of(n, masked, dtype, seed):
    cache, kv = states([n, 130], 2, dtype, seed)
    k, v = kv[0]
    k = k.clone()
    k[masked, 1, 5] = -INF
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[masked] = False
    return cache, kv, keep


def check(out, q, kv, keep, g):
    """Rows of the sequence with masked keys: KV head 0 as ever, KV head 1 over the keys left."""
    k, v = kv
    ref.assert_close(out[:, :g], *ref.attention(q[:, :g], k[:, :1], v[:, :1]))
    ref.assert_close(out[:, g:], *ref.attention(q[:, g:], k[keep, 1:], v[keep, 1:]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("g", [3, 8, 12])
@pytest.mark.parametrize("n,masked", CASES)
def test_decode_gives_a_score_of_minus_infinity_no_weight(n, masked, g, dtype):
    cache, kv, keep = cache_of(n, masked, dtype, 11)
    q = queries(2, 2 * g, dtype, 12)
    out = decode(cache, 1, q, [n, 130])
    check(out[:1], q[:1], kv[0], keep, g)
    ref.assert_close(out[1:], *ref.attention(q[1:], *kv[1]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 20, 128, 300, 9000])
@pytest.mark.parametrize("value", [-INF, INF])
def test_decode_rows_without_a_softmax_are_nan_and_alone(n, value, dtype):
    g = 4
    cache, kv = states([n, 130], 2, dtype, 15)
    k, v = kv[0]
    k = k.clone()
    k[:, 1, 5] = -INF                   # every score of KV head 1 is -inf ..
    if value == INF:
        k[n // 2, 1, 5] = INF           # .. but for one of +inf
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = queries(2, 2 * g, dtype, 16)
    out = decode(cache, 1, q, [n, 130])
    assert out[0, g:].isnan().all()
    ref.assert_close(out[:1, :g], *ref.attention(q[:1, :g], k[:, :1], v[:, :1]))
    ref.assert_close(out[1:], *ref.attention(q[1:], *kv[1]))


@pytest.mark.parametrize("dtype", TYPES)
def test_decode_heads_of_one_kv_head_that_score_differently(dtype):
    n, g = 200, 8
    cache, kv = states([n, 130], 2, dtype, 17)
    k, v = kv[0]
    k = k.clone()
    k[:100, 1, 5] = -INF
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = queries(2, 2 * g, dtype, 18)
    q[:, 1::2, 5] *= -1.0
    keep = torch.arange(n, device="cuda") >= 100
    out = decode(cache, 1, q, [n, 130])[:1]
    assert out[:, g + 1::2].isnan().all()
    ref.assert_close(out[:, :g:2], *ref.attention(q[:1, :g:2], k[:, :1], v[:, :1]))
    ref.assert_close(out[:, g::2], *ref.attention(q[:1, g::2], k[keep, 1:], v[keep, 1:]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,g", [(1, 3), (2, 12), (40, 4), (130, 4)])
@pytest.mark.parametrize("n,masked", CASES)
def test_cross_gives_a_score_of_minus_infinity_no_weight(n, masked, rows, g, dtype):
    cache, kv, keep = cache_of(n, masked, dtype, 13)
    q = queries(rows + 3, 2 * g, dtype, 14)
    out = cross(cache, 1, q, [rows, 3], [n, 130])
    check(out[:rows], q[:rows], kv[0], keep, g)
    ref.assert_close(out[rows:], *ref.attention(q[rows:], *kv[1]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 20, 128, 300, 9000])
@pytest.mark.parametrize("value", [-INF, INF])
def test_cross_rows_without_a_softmax_are_nan_and_alone(n, value, dtype):
    g = 4
    cache, kv = states([n, 130], 2, dtype, 15)
    k, v = kv[0]
    k = k.clone()
    k[:, 1, 5] = -INF                   # every score of KV head 1 is -inf ..
    if value == INF:
        k[n // 2, 1, 5] = INF           # .. but for one of +inf
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = queries(43, 2 * g, dtype, 16)
    out = cross(cache, 1, q, [40, 3], [n, 130])
    assert out[:40, g:].isnan().all()
    ref.assert_close(out[:40, :g], *ref.attention(q[:40, :g], k[:, :1], v[:, :1]))
    ref.assert_close(out[40:], *ref.attention(q[40:], *kv[1]))


@pytest.mark.parametrize("dtype", TYPES)
def test_cross_heads_of_one_kv_head_that_score_differently(dtype):
    # the same infinite key is -inf for one query head, +inf for the next
    n, g = 200, 8
    cache, kv = states([n, 130], 2, dtype, 17)
    k, v = kv[0]
    k = k.clone()
    k[:100, 1, 5] = -INF
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = queries(30, 2 * g, dtype, 18)
    q[:, 1::2, 5] *= -1.0
    keep = torch.arange(n, device="cuda") >= 100
    out, r = cross(cache, 1, q, [27, 3], [n, 130])[:27], q[:27]
    assert out[:, g + 1::2].isnan().all()
    ref.assert_close(out[:, :g], *ref.attention(r[:, :g], k[:, :1], v[:, :1]))
    ref.assert_close(out[:, g::2], *ref.attention(r[:, g::2], k[keep, 1:], v[keep, 1:]))


def test_cross_keys_of_minus_infinity_shield_the_largest_values():
    # a weight of zero times the type's largest value is zero, not a rest of the exponential
    n, g = 200, 4
    cache, kv, keep = cache_of(n, list(range(40, 180)), torch.bfloat16, 19)
    k, v = kv[0]
    v = v.clone()
    v[~keep, 1] = torch.finfo(torch.bfloat16).max
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    cache.pool[1][cache.block_table[0].long()[torch.arange(40, 180) // 128], 1, 0, torch.arange(40, 180) % 128, 5] = -INF
    q = queries(9, 2 * g, torch.bfloat16, 20)
    check(cross(cache, 1, q, [6, 3], [n, 130])[:6], q[:6], (k, v), keep, g)
