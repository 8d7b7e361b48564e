"""The calls around the cache on the GPU against plain 64-bit references: step tables, rotary
rows, raw pages and the two attention calls over them, alone and as one serving step."""

import math
import random

import numpy as np
import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests import gpu_helpers as gh
from tests import serving_reference as ref

pytestmark = pytest.mark.gpu
P, D = 128, 128
TYPES = [torch.bfloat16, torch.float16]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ step tables
def run_tables(cached, new, ring, state, table, rows, in_place=False, ws=None):
    d = dict(cached=i32(cached), new=i32(new), ring=i32(ring), state=i32(state), table=i32(table))
    n = len(cached)
    seq = d["cached"] if in_place else torch.full((n,), -7, dtype=torch.int32, device="cuda")
    out = d["state"] if in_place else torch.full((2,), -7, dtype=torch.int32, device="cuda")
    cu = torch.full((n + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((rows,), -7, dtype=torch.int64, device="cuda")
    pos = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    ws = torch.zeros(4, dtype=torch.int32, device="cuda") if ws is None else ws
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvtc.kvtc_step_tables(d["cached"], d["new"], d["ring"], d["state"], d["table"], seq, cu, slots, pos, out, ws,
                          status)
    torch.cuda.synchronize()
    assert ws.abs().sum().item() == 0
    return dict(ring=d["ring"].cpu().numpy(), state=out.tolist(), table=d["table"].cpu().numpy(),
                seq_lens=seq.cpu().numpy(), cu=cu.cpu().numpy(), slots=slots.cpu().numpy(),
                positions=pos.cpu().numpy(), status=status.item())


def tables_case(seed, n_seq, top_cached, top_new, max_pages, spare, rows_extra, odd=False):
    r = random.Random(seed)
    cached = [r.choice([0, r.randint(0, top_cached), 128 * r.randint(0, top_cached // 128)]) for _ in range(n_seq)]
    new = [r.choice([-1, 0, 1, 1, r.randint(0, top_new)]) for _ in range(n_seq)]
    if odd:  # lengths out of range, tokens beyond the table
        for s in range(0, n_seq, 5):
            cached[s] = r.choice([-1, -(1 << 31), max_pages * P + 1, (1 << 31) - 1, max_pages * P])
        for s in range(1, n_seq, 7):
            new[s] = r.choice([(1 << 31) - 1, max_pages * P, -(1 << 31)])
    held = [ref.pages(c) if 0 <= c <= max_pages * P else 0 for c in cached]
    total = sum(held) + spare
    ids = list(range(total))
    r.shuffle(ids)
    table = np.full((n_seq, max_pages), -1, np.int32)
    for s, h in enumerate(held):
        table[s, :h] = [ids.pop() for _ in range(h)]
    capacity = total + r.randint(1, 5)
    head = r.randrange(capacity)
    ring = np.full(capacity, -1, np.int32)
    for i, p in enumerate(ids):
        ring[(head + i) % capacity] = p
    rows = sum(n for n in new if 0 < n < 100000) + rows_extra
    return cached, new, ring, [head, len(ids)], table, max(0, rows)


def same_tables(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_seq,top_cached,top_new,spare,extra", [
    (1, 5, 1, 3, 0), (3, 700, 1, 9, 2), (33, 1000, 300, 200, 17), (5, 0, 0, 4, 0), (40, 900, 260, 20, 5),
    (1024, 400, 3, 3000, 0), (1025, 400, 20, 3000, 9), (2500, 300, 40, 2000, 100), (7, 800, 3000, 500, -2000)])
def test_step_tables(n_seq, top_cached, top_new, spare, extra, in_place):
    case = tables_case(n_seq * 7 + spare, n_seq, top_cached, top_new, 32, spare, extra)
    same_tables(run_tables(*case, in_place=in_place), ref.step_tables(*case))


@pytest.mark.parametrize("seed", range(4))
def test_step_tables_with_lengths_out_of_range(seed):
    case = tables_case(seed, 60, 500, 200, 5, 60, 11, odd=True)
    got, want = run_tables(*case), ref.step_tables(*case)
    assert want["status"] & 2
    same_tables(got, want)


def test_step_tables_refuse_pages_that_are_not_there():
    # 3 free pages: the first sequence takes 2, the second lacks 2, the third needs none
    table = np.array([[-1, -1, -1, -1], [9, -1, -1, -1], [8, -1, -1, -1], [-1, -1, -1, -1]], np.int32)
    case = ([0, 128, 100, 0], [200, 200, 28, 1], [5, 6, 7, -1], [0, 3], table, 500)
    got, want = run_tables(*case), ref.step_tables(*case)
    same_tables(got, want)
    assert got["status"] == kvtc.STATUS_NO_PAGE
    assert got["seq_lens"].tolist() == [200, 128, 128, 0]
    assert got["state"] == [2, 1]


def test_step_tables_report_bad_rings_and_pages():
    table = np.full((2, 3), -1, np.int32)
    for state in ([4, 0], [-1, 2], [0, 5], [0, -1]):
        case = ([0, 130], [1, -1], [1, 2, 3, 0], state, table, 4)
        got = run_tables(*case)
        same_tables(got, ref.step_tables(*case))
        assert got["status"] & kvtc.STATUS_BAD_PAGE
    # a full ring cannot take pages back; a negative id in the table gives no slot
    case = ([130, 5], [-1, 3], [1, 2, 3, 0], [1, 4], np.array([[7, 8, -1], [-3, -1, -1]], np.int32), 4)
    got = run_tables(*case)
    same_tables(got, ref.step_tables(*case))
    assert got["status"] & kvtc.STATUS_BAD_PAGE and got["slots"].tolist() == [-1] * 4


def test_step_tables_many_rows_and_no_rows():
    case = tables_case(5, 300, 2000, 900, 64, 4000, 50000)
    assert case[5] > 3 * 4096
    ws = torch.zeros(4, dtype=torch.int32, device="cuda")
    for _ in range(3):
        same_tables(run_tables(*case, in_place=True, ws=ws), ref.step_tables(*case))
    cached, new, ring, state, table, _ = tables_case(6, 20, 500, 1, 8, 30, 0)
    case = (cached, [-1 if n else 0 for n in new], ring, state, table, 0)
    same_tables(run_tables(*case), ref.step_tables(*case))


def test_step_tables_loop_replayed_from_a_graph():
    # lengths and ring state in place: five replays are five steps
    cached, new, ring, state, table, _ = tables_case(8, 12, 300, 60, 32, 200, 0)
    new = [abs(n) for n in new]
    rows = sum(new) + 3
    want = (cached, ring, state, table)
    lens, fresh, ring_d, st, tab = i32(cached), i32(new), i32(ring), i32(state), i32(table)
    cu, slots = torch.empty(13, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda")
    pos, ws = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvtc.kvtc_step_tables(lens, fresh, ring_d, st, tab, lens, cu, slots, pos, st, ws)
    for _ in range(5):
        g.replay()
        w = ref.step_tables(want[0], new, want[1], want[2], want[3], rows)
        want = (w["seq_lens"].tolist(), w["ring"], w["state"], w["table"])
        torch.cuda.synchronize()
        assert lens.tolist() == want[0] and st.tolist() == want[2]
        assert np.array_equal(slots.cpu().numpy(), w["slots"]) and np.array_equal(tab.cpu().numpy(), w["table"])


# ------------------------------------------------------------------ rotary rows
def rows(n, heads, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads + pad, D), generator=g).to(dtype).cuda()
    return x[:, :heads]


def positions(n_axes, n, seed, top=100000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, top, (n_axes, n), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32] + TYPES)
@pytest.mark.parametrize("n,hq,hk,sections,interleaved,pad", [
    (1, 1, 1, (64,), False, 0), (3, 32, 8, (16, 24, 24), False, 0), (5, 28, 4, (24, 20, 20), True, 8),
    (130, 7, 7, (0, 1, 63), True, 1), (17, 200, 3, (10, 20, 30, 4), False, 3), (1000, 2, 1, (32, 32), True, 0)])
def test_rope(n, hq, hk, sections, interleaved, pad, dtype):
    q, k = rows(n, hq, dtype, 1, pad), rows(n, hk, dtype, 2, pad)
    pos = positions(len(sections), n, 3)
    d = kvtc.rope_desc(sections, interleaved)
    for inverse in (False, True):
        qo, ko = torch.empty(q.shape, dtype=dtype, device="cuda"), torch.empty(k.shape, dtype=dtype, device="cuda")
        kvtc.kvtc_rope(d, q, k, pos, qo, ko, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            want = ref.rope(x, pos, sections, interleaved, inverse=inverse)
            ref.assert_close(y, want, ref.rope_bound(x, dtype))


def test_rope_in_place_alone_and_far_positions():
    # 2^31 - 1: the product of position and frequency is rounded in 64 bits on both sides
    # (2^-53 of 2^31 rad each), far above the fp32 bound's share of the angle
    q, k = rows(9, 4, torch.float32, 4), rows(9, 2, torch.float32, 5)
    pos = i32([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 77, 131071, 5])
    d = kvtc.rope_desc([64], base=10000.0)
    want_q, want_k = (ref.rope(x, pos, [64], base=10000.0) for x in (q, k))
    qi = q.clone()
    kvtc.kvtc_rope(d, qi, None, pos, qi, None)
    ref.assert_close(qi, want_q, ref.rope_bound(q, torch.float32, far=4.0))
    ki = k.clone()
    kvtc.kvtc_rope(d, None, ki, pos, None, ki)
    ref.assert_close(ki, want_k, ref.rope_bound(k, torch.float32, far=4.0))
    assert torch.equal(qi[0], q[0])                    # position 0 does not turn


def test_rope_inverse_is_the_gradient():
    # <w, R x> has gradient R^T w in x: against the 64-bit formula's and against differences
    n, h, sections = 6, 3, (16, 24, 24)
    x, w, pos = rows(n, h, torch.float32, 6), rows(n, h, torch.float32, 7), positions(3, n, 8)
    d = kvtc.rope_desc(sections)
    grad = torch.empty_like(w)
    kvtc.kvtc_rope(d, w, None, pos, grad, None, inverse=True)
    leaf = x.double().requires_grad_()
    (ref.rope(leaf, pos, sections) * w.double()).sum().backward()
    ref.assert_close(grad, leaf.grad, ref.rope_bound(w, torch.float32))
    y0, y1, step = torch.empty_like(x), torch.empty_like(x), 2.0 ** -3
    for t, a, i in ((0, 0, 0), (2, 1, 63), (5, 2, 100)):
        e = torch.zeros_like(x)
        e[t, a, i] = step
        kvtc.kvtc_rope(d, x + e, None, pos, y1, None)
        kvtc.kvtc_rope(d, x - e, None, pos, y0, None)
        slope = (((y1.double() - y0.double()) * w.double()).sum() / (2 * step)).item()
        # linear: the differences' rounding is 2 values of at most |x| ~ 5 by 14 * 2^-24, on
        # two elements of w, over the step
        assert abs(slope - grad[t, a, i].item()) <= 2 * 2 * 10 * 14 * 2.0 ** -24 * 5 / (2 * step)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,hq,hk,sections,pad", [(1, 4, 1, (64,), 0), (37, 28, 4, (16, 24, 24), 0),
                                                  (300, 32, 8, (24, 40), 8), (19, 0, 20, None, 2)])
def test_raw_append(n, hq, hk, sections, pad, dtype):
    k, v = rows(n, hk, dtype, 1, pad), rows(n, hk, dtype, 2, pad)
    n_pages = 9
    cache = kvtc.RawCache(3, hk, n_pages, torch.zeros((1, 1), dtype=torch.int32), dtype=dtype)
    cache.pool.copy_(torch.randn(cache.pool.shape, dtype=torch.float32, device="cuda"))
    before = cache.pool.clone()
    r = np.random.default_rng(n)
    slots = r.permutation(n_pages * P)[:n].astype(np.int64)
    bad = []
    if n > 10:
        slots[3], slots[7], slots[9] = -1, n_pages * P, (1 << 62)
        bad = [3, 7, 9]
    good = [i for i in range(n) if i not in bad]
    slots_d = torch.from_numpy(slots).cuda()
    if sections is None:
        kvtc.kvtc_raw_append(cache, 2, k, v, slots_d)
    else:
        q, pos = rows(n, hq, dtype, 3, pad), positions(len(sections), n, 4)
        qo = torch.empty(q.shape, dtype=dtype, device="cuda")
        kvtc.kvtc_raw_append(cache, 2, k, v, slots_d, rope=kvtc.rope_desc(sections), positions=pos, q=q, q_out=qo)
        ref.assert_close(qo, ref.rope(q, pos, sections), ref.rope_bound(q, dtype))
    assert cache.status.item() == (kvtc.STATUS_BAD_PAGE if bad else 0)
    page, row = slots_d[good] // P, slots_d[good] % P
    assert torch.equal(cache.pool[2][page, :, 1, row], v[good])
    got = cache.pool[2][page, :, 0, row].clone()
    if sections is None:
        assert torch.equal(got, k[good])
    else:
        ref.assert_close(got, ref.rope(k, pos, sections)[good], ref.rope_bound(k, dtype)[good])
        only_k = kvtc.RawCache(3, hk, n_pages, torch.zeros((1, 1), dtype=torch.int32), dtype=dtype)
        kvtc.kvtc_raw_append(only_k, 2, k, v, slots_d, rope=kvtc.rope_desc(sections), positions=pos)
        assert torch.equal(only_k.pool[2][page, :, 0, row], got)
    after = cache.pool.clone()
    after[2][page, :, :, row] = before[2][page, :, :, row]
    assert torch.equal(after, before)                  # nothing else was touched


# ------------------------------------------------------------------ attention
def states(lens, hk, dtype, seed, n_layers=2, layer=1, garbage=float("nan"), max_pages=None):
    """A cache whose unwritten slots hold garbage, and each sequence's K and V."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max_pages or max(1, max(ref.pages(n) for n in lens))
    n_pages = sum(ref.pages(n) for n in lens) + 2
    ids = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(lens), max_pages), -5, np.int32)
    at = 0
    for s, n in enumerate(lens):
        table[s, :ref.pages(n)] = ids[at:at + ref.pages(n)]
        at += ref.pages(n)
    cache = kvtc.RawCache(n_layers, hk, n_pages, torch.from_numpy(table), dtype=dtype)
    cache.pool.fill_(garbage)
    kv = []
    for s, n in enumerate(lens):
        k = torch.randn((n, hk, D), generator=g).to(dtype).cuda()
        v = torch.randn((n, hk, D), generator=g).to(dtype).cuda()
        ref.scatter_states(cache.pool, layer, cache.block_table, s, k, v)
        kv.append((k, v))
    return cache, kv


def decode(cache, layer, q, lens, max_len=None, scale=0.0, ws=None):
    n_seq, hq = q.shape[:2]
    max_len = max(lens) if max_len is None else max_len
    if ws is None:
        ws = torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(n_seq, hq, cache.n_kv_heads, max_len), dtype=torch.uint8,
                         device="cuda")
    out = torch.full_like(q, float("nan"))
    kvtc.kvtc_raw_decode_attention(cache, layer, q, i32(lens), max_len, out, ws, scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,hq,hk", [
    ([1], 1, 1), ([0], 4, 2), ([128], 4, 1), ([129, 127], 8, 2), ([1, 2, 15, 16, 17, 63, 64, 65, 0, 300], 28, 4),
    ([1000, 0, 517], 32, 8), ([5000], 7, 1), ([20000, 3], 40, 2), ([2049] * 3, 64, 1), ([700, 40], 20, 20),
    ([333, 90], 24, 2), ([260], 256, 1), ([130] * 70, 3, 3)])
def test_raw_decode(lens, hq, hk, dtype):
    cache, kv = states(lens, hk, dtype, 11)
    q = (torch.randn((len(lens), hq, D), generator=torch.Generator().manual_seed(2)) * 1.5).to(dtype).cuda()
    out = decode(cache, 1, q, lens)
    assert cache.status.item() == 0
    for s, (k, v) in enumerate(kv):
        want, bound = ref.attention(q[s:s + 1], k, v)
        ref.assert_close(out[s:s + 1], want, bound)


@pytest.mark.parametrize("garbage", [float("inf"), -float("inf"), -65504.0])
def test_raw_decode_ignores_what_unwritten_slots_hold(garbage):
    lens = [3, 130, 64, 199]
    cache, kv = states(lens, 2, torch.float16, 5, garbage=garbage)
    q = torch.randn((4, 6, D), generator=torch.Generator().manual_seed(3)).half().cuda()
    out = decode(cache, 1, q, lens)
    for s, (k, v) in enumerate(kv):
        ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], k, v))


def test_raw_decode_scale_sharp_and_flat():
    lens = [3000, 77]
    cache, kv = states(lens, 2, torch.bfloat16, 6)
    q = torch.randn((2, 8, D), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    for scale in (2.0, 1e-6):
        out = decode(cache, 1, q, lens, scale=scale)
        for s, (k, v) in enumerate(kv):
            ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], k, v, scale))


def test_raw_decode_reports_bad_lengths_and_pages_and_goes_on():
    lens = [300, 200, 400, 500, 129]
    cache, kv = states(lens, 2, torch.bfloat16, 7)
    q = torch.randn((5, 8, D), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    out = decode(cache, 1, q, [300, -1, 400, 501, 129], max_len=500)
    assert cache.status.item() == kvtc.STATUS_BAD_POS
    assert not out[1].any() and not out[3].any()
    for s in (0, 2, 4):
        ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], *kv[s]))
    cache.status.zero_()
    n_pages = cache.desc.n_pages
    cache.block_table[0, 1], cache.block_table[2, 3], cache.block_table[4, 1] = -1, n_pages, 1 << 30
    ws = torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(5, 8, 2, 500), dtype=torch.uint8, device="cuda")
    out = decode(cache, 1, q, lens, ws=ws)
    assert cache.status.item() == kvtc.STATUS_BAD_PAGE
    assert not out[0].any() and not out[2].any() and not out[4].any()
    for s in (1, 3):
        ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], *kv[s]))
    # the workspace serves the next call
    cache.status.zero_()
    out = decode(cache, 1, q, [100, 200, 300, 500, 100], ws=ws)
    assert cache.status.item() == 0
    for s, n in enumerate([100, 200, 300, 500, 100]):
        ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], kv[s][0][:n], kv[s][1][:n]))


def test_raw_decode_is_the_same_every_time_and_under_a_looser_bound():
    lens = [9000, 1, 2500, 4097]
    cache, kv = states(lens, 4, torch.bfloat16, 8, max_pages=200)
    q = torch.randn((4, 16, D), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    first = decode(cache, 1, q, lens)
    for _ in range(5):
        assert torch.equal(decode(cache, 1, q, lens), first)
    out = decode(cache, 1, q, lens, max_len=200 * P)   # another split
    for s, (k, v) in enumerate(kv):
        ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], k, v))


def cross(cache, layer, q, q_lens, lens, max_len=None, scale=0.0, ws=None, cu=None):
    n, hq = q.shape[:2]
    cu = np.concatenate([[0], np.cumsum(q_lens)]) if cu is None else cu
    max_len = max(lens) if max_len is None else max_len
    if ws is None:
        ws = torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(len(lens), n, hq, cache.n_kv_heads, max_len),
                         dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 123.0)
    kvtc.kvtc_raw_cross_attention(cache, layer, q, i32(cu), i32(lens), max_len, out, ws, scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,lens,hq,hk", [
    ([1], [1], 1, 1), ([5], [0], 4, 2), ([64], [128], 4, 1), ([33, 0, 7], [129, 127, 64], 8, 2),
    ([4, 1, 17], [1501, 700, 1500], 20, 20), ([300], [3000], 7, 1), ([129, 260, 1], [257, 0, 900], 28, 4),
    ([3], [20000], 40, 2), ([50, 2], [300, 200], 128, 1), ([200], [555], 24, 2), ([3] * 40, [140] * 40, 3, 3),
    ([1000], [1], 2, 2)])
def test_raw_cross(q_lens, lens, hq, hk, dtype):
    cache, kv = states(lens, hk, dtype, 21)
    n = sum(q_lens)
    q = (torch.randn((n, hq, D), generator=torch.Generator().manual_seed(7)) * 1.5).to(dtype).cuda()
    out = cross(cache, 1, q, q_lens, lens)
    assert cache.status.item() == 0
    at = 0
    for (k, v), m in zip(kv, q_lens):
        ref.assert_close(out[at:at + m], *ref.attention(q[at:at + m], k, v))
        at += m


@pytest.mark.parametrize("garbage", [float("inf"), -float("inf"), -65504.0])
def test_raw_cross_ignores_what_unwritten_slots_hold(garbage):
    q_lens, lens = [40, 5, 90], [3, 130, 199]
    cache, kv = states(lens, 2, torch.float16, 5, garbage=garbage)
    q = torch.randn((135, 6, D), generator=torch.Generator().manual_seed(3)).half().cuda()
    out = cross(cache, 1, q, q_lens, lens)
    at = 0
    for (k, v), m in zip(kv, q_lens):
        ref.assert_close(out[at:at + m], *ref.attention(q[at:at + m], k, v))
        at += m


def test_raw_cross_growing_scores_and_scales():
    # keys whose scores keep growing along the sequence: the running maximum moves on
    lens, n = [2000], 150
    cache, kv = states(lens, 1, torch.bfloat16, 9)
    ramp = torch.linspace(0.0, 6.0, 2000, device="cuda").view(-1, 1, 1)
    k = (kv[0][0].float() * ramp).bfloat16()
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, kv[0][1])
    q = torch.randn((n, 4, D), generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    for scale in (0.0, 0.5, 1e-6):
        out = cross(cache, 1, q, [n], lens, scale=scale)
        ref.assert_close(out, *ref.attention(q, k, kv[0][1], scale or 1 / math.sqrt(D)))
    out = decode(cache, 1, q[:1], lens, scale=0.5)
    ref.assert_close(out, *ref.attention(q[:1], k, kv[0][1], 0.5))


def test_raw_cross_leaves_rows_outside_and_reports_bad_rows_and_pages():
    lens = [300, 200, 400]
    cache, kv = states(lens, 2, torch.bfloat16, 10)
    q = torch.randn((100, 8, D), generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    out = cross(cache, 1, q, None, lens, cu=[5, 30, 31, 90])
    assert cache.status.item() == 0
    assert (out[:5] == 123.0).all() and (out[90:] == 123.0).all()
    for s, (a, b) in enumerate(((5, 30), (30, 31), (31, 90))):
        ref.assert_close(out[a:b], *ref.attention(q[a:b], *kv[s]))
    out = cross(cache, 1, q, None, lens, cu=[0, 30, 40, 101])       # beyond the rows: skipped
    assert cache.status.item() == kvtc.STATUS_BAD_POS and (out[40:] == 123.0).all()
    ref.assert_close(out[:30], *ref.attention(q[:30], *kv[0]))
    ref.assert_close(out[30:40], *ref.attention(q[30:40], *kv[1]))
    cache.status.zero_()
    out = cross(cache, 1, q, None, [300, 200, 401], max_len=400, cu=[0, 30, 40, 100])
    assert cache.status.item() == kvtc.STATUS_BAD_POS and not out[40:].any()
    cache.status.zero_()
    cache.block_table[0, 2], cache.block_table[2, 0] = -1, cache.desc.n_pages
    ws = torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(3, 100, 8, 2, 400), dtype=torch.uint8, device="cuda")
    out = cross(cache, 1, q, [30, 10, 60], lens, ws=ws)
    assert cache.status.item() == kvtc.STATUS_BAD_PAGE and not out[:30].any() and not out[40:].any()
    ref.assert_close(out[30:40], *ref.attention(q[30:40], *kv[1]))
    cache.status.zero_()
    out = cross(cache, 1, q, [30, 10, 60], [256, 200, 0], ws=ws)    # the workspace serves the next call
    assert cache.status.item() == 0 and not out[40:].any()
    ref.assert_close(out[:30], *ref.attention(q[:30], kv[0][0][:256], kv[0][1][:256]))


def test_raw_cross_is_the_same_every_time():
    q_lens, lens = [100, 700, 3], [9000, 300, 2500]
    cache, _ = states(lens, 4, torch.bfloat16, 8)
    q = torch.randn((803, 16, D), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    first = cross(cache, 1, q, q_lens, lens)
    for _ in range(5):
        assert torch.equal(cross(cache, 1, q, q_lens, lens), first)


def test_offsets_beyond_32_bits():
    # a pool whose last page starts beyond 2^32 bytes (and 2^31 elements)
    hk = 8
    n_pages = (1 << 32) // (hk * 2 * P * D * 2) + 40
    cache = kvtc.RawCache(1, hk, n_pages, torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32))
    k, v = rows(200, hk, torch.bfloat16, 1), rows(200, hk, torch.bfloat16, 2)
    t = torch.arange(200, device="cuda")
    slots = cache.block_table[0].long()[t // P] * P + t % P
    kvtc.kvtc_raw_append(cache, 0, k, v, slots)
    q = rows(40, 16, torch.bfloat16, 3).contiguous()
    ref.assert_close(decode(cache, 0, q[:1].contiguous(), [200]), *ref.attention(q[:1], k, v))
    ref.assert_close(cross(cache, 0, q, [40], [200]), *ref.attention(q, k, v))


# ------------------------------------------------------------------ together
def test_a_serving_loop_of_all_calls():
    """Requests come, grow token by token, one finishes and its pages serve another; layer 0
    is coded (kvtc_encode_append / kvtc_decode_attention), layer 1 raw with three position
    axes; the loop runs on a side stream.  Every step's tables are those of the reference,
    both layers' outputs match."""
    hk, g, n_seq, max_pages, n_pages = 2, 4, 3, 6, 14
    hq = hk * g
    r = np.random.default_rng(3)
    plan = gh.random_plan(1, hk, g, [((64, 4), (64, 4))] * hk, r)
    table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
    coded = kvtc.Cache(plan, n_pages, table)
    rawc = kvtc.RawCache(2, hk, n_pages, table)
    assert rawc.block_table.data_ptr() == table.data_ptr() == coded.block_table.data_ptr()
    ring, state = torch.arange(n_pages, dtype=torch.int32, device="cuda"), i32([0, n_pages])
    lens, ws = i32([0] * n_seq), torch.zeros(4, dtype=torch.int32, device="cuda")
    seq, state_out = torch.empty_like(lens), torch.empty_like(state)
    cu = torch.empty(n_seq + 1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sections, desc = (16, 24, 24), kvtc.rope_desc((16, 24, 24))
    max_len = max_pages * P
    ws_c = torch.zeros(kvtc.kvtc_decode_workspace_bytes(plan, n_seq, max_len), dtype=torch.uint8, device="cuda")
    ws_r = torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(n_seq, hq, hk, max_len), dtype=torch.uint8, device="cuda")
    ws_x = torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(n_seq, 700, hq, hk, max_len), dtype=torch.uint8, device="cuda")
    raw_kv = [[torch.zeros((0, hk, D), dtype=torch.bfloat16, device="cuda")] * 2 for _ in range(n_seq)]
    want = dict(seq_lens=np.zeros(n_seq, np.int32), ring=np.arange(n_pages), state=[0, n_pages],
                table=table.cpu().numpy())
    coded_kv = [[np.zeros((0, hk, D), np.float32)] * 2 for _ in range(n_seq)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step, new in enumerate([[300, 127, 0], [1, 1, 40], [1, 1, 1], [1, -1, 1], [1, 0, 1], [1, 500, 1], [1, 1, 1]]):
        n_rows = sum(max(n, 0) for n in new) + 2       # two padding rows
        slots, pos = torch.empty(n_rows, dtype=torch.int64, device="cuda"), torch.empty(n_rows, dtype=torch.int32, device="cuda")
        x = torch.from_numpy(r.standard_normal((n_rows, hq + 2 * hk, D)).astype(np.float32)).bfloat16().cuda()
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        q_rot = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        outs = [torch.full((n_seq, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out_x = torch.full((n_rows, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        fresh = i32(new)
        kc, vc = k.contiguous(), v.contiguous()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            kvtc.kvtc_step_tables(lens, fresh, ring, state, table, seq, cu, slots, pos, state_out, ws, status)
            pos3 = torch.stack([pos, pos // 2, pos + 3]).contiguous()
            n_new = n_rows - 2
            if n_new:
                kvtc.kvtc_encode_append(plan, coded, 0, kc[:n_new], vc[:n_new], cu, lens)
            kvtc.kvtc_raw_append(rawc, 1, k, v, slots, rope=desc, positions=pos3, q=q, q_out=q_rot)
            last = (cu[1:].long() - 1).clamp(min=0)
            q_last = q_rot[last].contiguous()
            kvtc.kvtc_decode_attention(plan, coded, 0, q_last, seq, max_len, outs[0], ws_c)
            kvtc.kvtc_raw_decode_attention(rawc, 1, q_last, seq, max_len, outs[1], ws_r)
            kvtc.kvtc_raw_cross_attention(rawc, 1, q_rot, cu, seq, max_len, out_x, ws_x)
        stream.synchronize()
        want = ref.step_tables(want["seq_lens"].tolist(), new, want["ring"], want["state"], want["table"], n_rows)
        assert want["status"] == status.item() == 0
        assert np.array_equal(table.cpu().numpy(), want["table"]) and state_out.tolist() == want["state"]
        assert np.array_equal(seq.cpu().numpy(), want["seq_lens"]) and np.array_equal(cu.cpu().numpy(), want["cu"])
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(pos.cpu().numpy(), want["positions"])
        live = slots.clamp(min=0)                      # (padding rows read some slot; they are not used)
        k_rot = rawc.pool[1][live // P, :, 0, live % P].clone()
        ref.assert_close(k_rot[:n_rows - 2], ref.rope(k, pos3, sections)[:n_rows - 2],
                         ref.rope_bound(k, torch.bfloat16)[:n_rows - 2])
        for s, n in enumerate(new):
            a, b = want["cu"][s], want["cu"][s + 1]
            if n < 0:
                raw_kv[s] = [k[:0], v[:0]]
                coded_kv[s] = [np.zeros((0, hk, D), np.float32)] * 2
            else:
                raw_kv[s] = [torch.cat([raw_kv[s][0], k_rot[a:b]]), torch.cat([raw_kv[s][1], v[a:b]])]
                coded_kv[s] = [np.concatenate([coded_kv[s][i], y[a:b].float().cpu().numpy()]) for i, y in enumerate((k, v))]
            ref.assert_close(outs[1][s:s + 1], *ref.attention(q_last[s:s + 1], *raw_kv[s]))
            ref.assert_close(out_x[a:b], *ref.attention(q_rot[a:b], *raw_kv[s]))
        assert (out_x[want["cu"][-1]:] == 9.0).all()
        seq_l = want["seq_lens"].tolist()
        o = gh.oracle_decode(plan, coded, 0, q_last.float().cpu().numpy(), seq_l, hk, g)
        got = outs[0].float().cpu().numpy()
        den = np.maximum(np.abs(o).max(-1, keepdims=True), 1e-30)
        assert (np.abs(got - o) <= (2e-3 + 2.0 ** -8) * den + 1e-30).all()
        if step == 0:
            assert gh.check_encode(plan, coded, 0, [tuple(c) for c in coded_kv], "bf16", hk) == 0
        lens.copy_(seq)
        state.copy_(state_out)
        torch.cuda.synchronize()
    assert rawc.status.item() == coded.status.item() == 0


def test_all_calls_in_one_graph_replayed_with_new_inputs():
    lens, q_lens, hq, hk = [700, 0, 1300], [30, 4, 200], 8, 2
    cache, kv = states(lens, hk, torch.bfloat16, 31)
    qd, qx = rows(3, hq, torch.bfloat16, 1).contiguous(), rows(234, hq, torch.bfloat16, 2).contiguous()
    sl, cu = i32(lens), i32([0, 30, 34, 234])
    ws_d = torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(3, hq, hk, 1300), dtype=torch.uint8, device="cuda")
    ws_x = torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(3, 234, hq, hk, 1300), dtype=torch.uint8, device="cuda")
    od, ox = torch.empty_like(qd), torch.empty_like(qx)
    qr = torch.empty_like(qd)
    pos = i32([5, 6, 7])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):  # two passes share the workspaces
            kvtc.kvtc_rope(kvtc.rope_desc([64]), qd, None, pos, qr, None)
            kvtc.kvtc_raw_decode_attention(cache, 1, qr, sl, 1300, od, ws_d)
            kvtc.kvtc_raw_cross_attention(cache, 1, qx, cu, sl, 1300, ox, ws_x)
    for seed in (5, 6):
        qd.copy_(rows(3, hq, torch.bfloat16, seed))
        qx.copy_(rows(234, hq, torch.bfloat16, seed + 10))
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for s, m in enumerate(q_lens):
            ref.assert_close(od[s:s + 1], *ref.attention(qr[s:s + 1], *kv[s]))
            ref.assert_close(ox[at:at + m], *ref.attention(qx[at:at + m], *kv[s]))
            at += m
