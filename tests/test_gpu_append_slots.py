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


# ------------------------------------------------------------------ rows placed by slot
@pytest.mark.parametrize("k_only", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_by_slot_are_the_codes_of_rows_by_position(dtype, k_only):
    plan, n_seq, n_pages = plan_of(3, k_only), 5, 23
    r = np.random.default_rng(4)
    table = torch.from_numpy(r.permutation(n_pages)[:n_seq * 4].reshape(n_seq, 4).astype(np.int32))
    start, new = [0, 127, 300, 5, 130], [200, 2, 40, 0, 250]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = rows(int(cu[-1]), dtype, 5)
    by_position, by_slot = kvtc.Cache(plan, n_pages, table), kvtc.Cache(plan, n_pages, table)
    for c in (by_position, by_slot):
        c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=torch.Generator().manual_seed(6), dtype=torch.uint8))
    kvtc.kvtc_encode_append(plan, by_position, 1, k, v, torch.from_numpy(cu).cuda(), torch.tensor(start, dtype=torch.int32).cuda())
    pos = np.concatenate([start[s] + np.arange(n) for s, n in enumerate(new)])
    seq = np.repeat(np.arange(n_seq), new)
    slots = table.numpy()[seq, pos // P].astype(np.int64) * P + pos % P
    # rows that go nowhere between the others, and rows beyond the pool
    order = r.permutation(len(slots) + 4)
    all_slots = np.concatenate([slots, [-1, -(1 << 62), n_pages * P, 1 << 62]])[order]
    pad = rows(4, dtype, 7)
    k2, v2 = (torch.cat([x, y])[torch.from_numpy(order).cuda()].contiguous() for x, y in zip((k, v), pad))
    kvtc.kvtc_encode_append_slots(plan, by_slot, 1, k2, v2, torch.from_numpy(all_slots).cuda())
    torch.cuda.synchronize()
    assert torch.equal(by_slot.pool, by_position.pool)
    assert by_position.status.item() == 0 and by_slot.status.item() == kvtc.STATUS_BAD_PAGE


@pytest.mark.parametrize("n_seq", [3, 140])
def test_a_sequence_without_pages_leaves_the_others_codes_alone(n_seq):
    """Row 0 finishes, row 1 takes its pages, and a new request comes to row 0, whose table row
    still names them, when the ring is empty: it is refused, in the middle of a replayed loop that
    reads no status.  Padding rows follow."""
    plan, max_pages = plan_of(8), 3
    n_pages = 2 + (n_seq - 1)                       # row 0 holds two pages, the others one each
    table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
    cache = kvtc.Cache(plan, n_pages, table)
    assert cache.block_table.data_ptr() == table.data_ptr()
    ring = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    state = torch.tensor([0, n_pages], dtype=torch.int32, device="cuda")
    lens, fresh = (torch.zeros(n_seq, dtype=torch.int32, device="cuda") for _ in range(2))
    n_rows = 340 + n_seq                            # (the first step has 325 + n_seq)
    cu = torch.empty(n_seq + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(n_rows, dtype=torch.int64, device="cuda")
    pos = torch.empty(n_rows, dtype=torch.int32, device="cuda")
    ws, status = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.empty((n_rows, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvtc.kvtc_step_tables(lens, fresh, ring, state, table, lens, cu, slots, pos, state, ws, status)
        kvtc.kvtc_encode_append_slots(plan, cache, 0, k, v, slots)
    kept = [[np.zeros((0, H, D), np.float32)] * 2 for _ in range(n_seq)]
    r = np.random.default_rng(9)
    ones = [1] * (n_seq - 2)
    for new, refused in (([200, 127] + ones, False), ([-1, 1] + ones, False), ([0, 129] + ones, False),
                         ([250, 1] + ones, True), ([0, 1] + ones, False), ([250, -1] + ones, True), ([250, 0] + ones, False)):
        fresh.copy_(torch.tensor(new, dtype=torch.int32))
        x = [r.standard_normal((n_rows, H, D)).astype(np.float32) for _ in range(2)]
        k.copy_(torch.from_numpy(x[0]))
        v.copy_(torch.from_numpy(x[1]))
        before = lens.tolist()
        g.replay()
        torch.cuda.synchronize()
        c, after = cu.tolist(), lens.tolist()
        assert (status.item() == kvtc.STATUS_NO_PAGE) == refused and status.item() in (0, kvtc.STATUS_NO_PAGE)
        status.zero_()
        for s, n in enumerate(new):
            if n < 0:
                assert after[s] == 0
                kept[s] = [np.zeros((0, H, D), np.float32)] * 2
            elif refused and s == 0:
                assert after[s] == before[s] and (slots[c[s]:c[s + 1]] == -1).all()
            else:
                assert after[s] == before[s] + n
                kept[s] = [np.concatenate([kept[s][i], y[c[s]:c[s + 1]].float().cpu().numpy()]) for i, y in enumerate((k, v))]
        # every code of every sequence is that of its own tokens (whole rows of codes: their
        # latents' bytes up to the sequence's last token)
        units = gh.plan_units(plan)
        for s in (0, 1, 2, n_seq - 1):
            t = len(kept[s][0])
            assert after[s] == t
            for u in range(2 * H):
                if t == 0:
                    continue
                got = gh.ocodec.unpack_sequence(gh.gpu_pages(cache, plan, u, s, -(-t // P)), u & 1, units[u]["r"], units[u]["b"], t)
                want = gh.oracle_codes(kept[s][u & 1][:, u >> 1], units[u], "bf16")
                assert np.array_equal(got, want), (s, u)
    assert cache.status.item() == 0


def test_rows_by_slot_refuse_what_does_not_fit():
    plan = plan_of(10)
    cache = kvtc.Cache(plan, 4, torch.zeros((1, 4), dtype=torch.int32))
    k, v = rows(3, torch.bfloat16, 11)
    slots = torch.arange(3, device="cuda")
    L, c = kvtc.lib(), kvtc.C.byref(cache.desc)
    p = lambda t: t.data_ptr()
    good = [plan.handle, c, 0, p(k), p(v), kvtc.KVTC_BF16, p(slots), 3, None]
    for i, bad in ((1, None), (2, -1), (2, 2), (3, None), (4, None), (5, kvtc.KVTC_F16), (5, 7), (6, None), (6, p(slots) + 4),
                   (7, -1)):
        a = list(good)
        a[i] = bad
        assert L.kvtc_encode_append_slots(*a) == 1, (i, bad)
    a = list(good)
    a[3] = a[4] = a[6] = None
    a[7] = 0
    assert L.kvtc_encode_append_slots(*a) == 0          # no rows
    no_table = kvtc.CacheDesc(cache.desc.pool, 4, None, 0, 0, cache.desc.status)
    assert L.kvtc_encode_append_slots(plan.handle, kvtc.C.byref(no_table), *good[2:]) == 0
    for change in (dict(slot_map=slots.int()), dict(slot_map=slots[:2]), dict(v=v[:2]), dict(v=v.float())):
        with pytest.raises(ValueError):
            kvtc.kvtc_encode_append_slots(plan, cache, 0, **dict(dict(k=k, v=v, slot_map=slots), **change))
    torch.cuda.synchronize()
    assert cache.status.item() == 0
