"""Edges of the calls around the cache on the GPU: units shared by many blocks, batches of many
sequences, values that are not finite, weights far below the maximum, shared workspaces, streams,
and drawn batches against the 64-bit references."""

import random

import numpy as np
import pytest
import torch

from bit_quantization_head_b200 import kvtc
from tests import serving_reference as ref
from tests.test_gpu_serving import cross, decode, i32, run_tables, same_tables, states, tables_case

pytestmark = pytest.mark.gpu
D = 128


def rand_q(n, hq, dtype, seed, scale=1.5):
    return (torch.randn((n, hq, D), generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def check_decode(cache, kv, q, lens, skip=(), **kw):
    out = decode(cache, 1, q, lens, **kw)
    for s, (k, v) in enumerate(kv):
        if s not in skip:
            ref.assert_close(out[s:s + 1], *ref.attention(q[s:s + 1], k, v))
    return out


def check_cross(cache, kv, q, q_lens, lens, skip=(), **kw):
    out = cross(cache, 1, q, q_lens, lens, **kw)
    at = 0
    for s, ((k, v), m) in enumerate(zip(kv, q_lens)):
        if s not in skip:
            ref.assert_close(out[at:at + m], *ref.attention(q[at:at + m], k, v))
        at += m
    return out


def decode_ws(n_seq, hq, hk, max_len):
    return torch.zeros(kvtc.kvtc_raw_decode_workspace_bytes(n_seq, hq, hk, max_len), dtype=torch.uint8, device="cuda")


def cross_ws(n_seq, n, hq, hk, max_len):
    return torch.zeros(kvtc.kvtc_raw_cross_workspace_bytes(n_seq, n, hq, hk, max_len), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ units shared by many blocks
@pytest.mark.parametrize("lens,hq,hk", [([50000], 3, 1), ([50000], 9, 1), ([40000, 100], 4, 2), ([30000, 0, 30000], 8, 4)])
def test_decode_of_long_sequences_joins_many_parts(lens, hq, hk):
    # more parts than are joined at once (48, and 128): groups of parts first
    cache, kv = states(lens, hk, torch.bfloat16, 41)
    q, ws = rand_q(len(lens), hq, torch.bfloat16, 42), decode_ws(len(lens), hq, hk, max(lens))
    first = check_decode(cache, kv, q, lens, ws=ws)
    assert not ws[:4096].any()
    assert torch.equal(decode(cache, 1, q, lens, ws=ws), first)
    # a bad page in the middle: zero, reported, and the counters are left for the next call
    page = cache.block_table[0, 150].item()
    cache.block_table[0, 150] = -2
    out = check_decode(cache, kv, q, lens, skip=(0,), ws=ws)
    assert cache.status.item() == kvtc.STATUS_BAD_PAGE and not out[0].any() and not ws[:4096].any()
    cache.block_table[0, 150] = page
    assert torch.equal(decode(cache, 1, q, lens, ws=ws), first)


@pytest.mark.parametrize("q_lens,lens,hq,hk", [([2], [40000], 4, 1), ([300], [20000], 4, 2), ([2, 65], [30000, 700], 2, 1)])
def test_cross_over_long_states_joins_parts(q_lens, lens, hq, hk):
    cache, kv = states(lens, hk, torch.bfloat16, 43)
    n = sum(q_lens)
    q, ws = rand_q(n, hq, torch.bfloat16, 44), cross_ws(len(lens), n, hq, hk, max(lens))
    first = check_cross(cache, kv, q, q_lens, lens, ws=ws)
    assert not ws[:4096].any()
    assert torch.equal(cross(cache, 1, q, q_lens, lens, ws=ws), first)
    page = cache.block_table[0, 100].item()
    cache.block_table[0, 100] = cache.desc.n_pages
    out = check_cross(cache, kv, q, q_lens, lens, skip=(0,), ws=ws)
    assert cache.status.item() == kvtc.STATUS_BAD_PAGE and not out[:q_lens[0]].any() and not ws[:4096].any()
    cache.block_table[0, 100] = page
    assert torch.equal(cross(cache, 1, q, q_lens, lens, ws=ws), first)


# ------------------------------------------------------------------ many sequences
def test_many_short_sequences():
    r = random.Random(5)
    lens = [r.choice([0, 1, 2, 5, 130]) for _ in range(700)]
    cache, kv = states(lens, 1, torch.float16, 45)
    q = rand_q(700, 2, torch.float16, 46)
    check_decode(cache, kv, q, lens)
    q_lens = [r.choice([0, 0, 1, 3]) for _ in range(700)]
    check_cross(cache, kv, rand_q(sum(q_lens), 2, torch.float16, 47), q_lens, lens)
    assert cache.status.item() == 0


def test_no_tokens_at_all():
    cache, _ = states([0, 0], 2, torch.bfloat16, 48)
    q = rand_q(2, 4, torch.bfloat16, 49)
    assert not decode(cache, 1, q, [0, 0], max_len=0).any()
    assert not cross(cache, 1, q, [1, 1], [0, 0], max_len=0).any()
    out = cross(cache, 1, q, [0, 0], [0, 0], max_len=0)
    assert (out == 123.0).all()                              # no sequence has rows
    assert cross(cache, 1, q[:0], [0, 0], [0, 0], max_len=0).shape[0] == 0


@pytest.mark.parametrize("seed", range(24))
def test_drawn_batches(seed):
    r = random.Random(1000 + seed)
    dtype = r.choice([torch.bfloat16, torch.float16])
    hk = r.choice([1, 2, 3, 5])
    g = r.choice([1, 2, 3, 4, 7, 8, 9, 12, 16, 17])
    n_seq = r.randint(1, 12)
    top = r.choice([1, 70, 300, 2500])
    lens = [r.choice([0, 1, r.randint(0, top), 128 * r.randint(0, max(1, top // 128))]) for _ in range(n_seq)]
    q_lens = [r.choice([0, 1, r.randint(1, 6), r.randint(1, 150)]) for _ in range(n_seq)]
    cache, kv = states(lens, hk, dtype, 50 + seed, max_pages=r.choice([None, 40]))
    check_decode(cache, kv, rand_q(n_seq, hk * g, dtype, seed, r.choice([0.1, 1.0, 4.0])), lens)
    check_cross(cache, kv, rand_q(sum(q_lens), hk * g, dtype, seed + 1, r.choice([0.1, 1.0, 4.0])), q_lens, lens)
    assert cache.status.item() == 0


# ------------------------------------------------------------------ values
def test_fp16_weights_far_below_the_maximum():
    # one key scores 14 above thousands of equal ones, whose weights of about 2^-20 make up
    # about a hundredth of the sum each thousand: they must not lose their bits
    n = 20000
    cache, kv = states([n], 1, torch.float16, 51)
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    k[777, 0, 0] = 14.0
    v = kv[0][1]
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, v)
    q = torch.zeros((130, 2, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    out = decode(cache, 1, q[:1], [n], scale=1.0)
    ref.assert_close(out, *ref.attention(q[:1], k, v, 1.0))
    out = cross(cache, 1, q, [130], [n], scale=1.0)
    ref.assert_close(out, *ref.attention(q, k, v, 1.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("token", [0, 1, 2, 3, 8, 9, 63, 64, 77, 129, 255])
def test_a_nan_among_the_keys_shows_in_its_heads_rows_only(token, dtype):
    lens, q_lens = [256, 200], [40, 30]
    cache, kv = states(lens, 2, dtype, 52)
    k = kv[0][0].clone()
    k[token, 1] = float("nan")
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, kv[0][1])
    q = rand_q(70, 8, dtype, 53)
    out = cross(cache, 1, q, q_lens, lens)
    assert out[:40, 4:].isnan().all()
    ref.assert_close(out[:40, :4], *ref.attention(q[:40, :4], kv[0][0][:, :1], kv[0][1][:, :1]))
    ref.assert_close(out[40:], *ref.attention(q[40:], *kv[1]))
    qd = torch.stack([q[0], q[40]])
    out = decode(cache, 1, qd, lens)
    assert out[0, 4:].isnan().all()
    ref.assert_close(out[:1, :4], *ref.attention(qd[:1, :4], kv[0][0][:, :1], kv[0][1][:, :1]))
    ref.assert_close(out[1:], *ref.attention(qd[1:], *kv[1]))


def test_scores_of_the_lowest_value_keep_their_order():
    # every score far below zero: nothing is special about the sign of the maximum
    lens = [300]
    cache, kv = states(lens, 1, torch.bfloat16, 54)
    k = -kv[0][0].float().abs().bfloat16() * 4
    ref.scatter_states(cache.pool, 1, cache.block_table, 0, k, kv[0][1])
    q = rand_q(140, 4, torch.bfloat16, 55).abs()
    ref.assert_close(cross(cache, 1, q, [140], lens), *ref.attention(q, k, kv[0][1]))
    ref.assert_close(decode(cache, 1, q[:1], lens), *ref.attention(q[:1], k, kv[0][1]))


# ------------------------------------------------------------------ workspaces, streams, graphs
def test_two_graphs_that_share_a_workspace_replayed_in_turn():
    hq, hk = 8, 2
    sizes = [([3000, 40], [100, 7]), ([500, 9000], [3, 300])]
    ws_d, ws_x = decode_ws(2, hq, hk, 9000), cross_ws(2, 400, hq, hk, 9000)
    graphs = []
    for i, (lens, q_lens) in enumerate(sizes):
        cache, kv = states(lens, hk, torch.bfloat16, 60 + i)
        qd, qx = rand_q(2, hq, torch.bfloat16, i), rand_q(sum(q_lens), hq, torch.bfloat16, 9 + i)
        od, ox, sl = torch.empty_like(qd), torch.empty_like(qx), i32(lens)
        cu = i32([0, q_lens[0], sum(q_lens)])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvtc.kvtc_raw_decode_attention(cache, 1, qd, sl, max(lens), od, ws_d)
            kvtc.kvtc_raw_cross_attention(cache, 1, qx, cu, sl, max(lens), ox, ws_x)
        graphs.append((g, cache, kv, qd, qx, od, ox, sl, cu))
    for i in (0, 1, 1, 0, 1):
        g, cache, kv, qd, qx, od, ox, *_ = graphs[i]
        od.fill_(float("nan"))
        ox.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for s, m in enumerate(sizes[i][1]):
            ref.assert_close(od[s:s + 1], *ref.attention(qd[s:s + 1], *kv[s]))
            ref.assert_close(ox[at:at + m], *ref.attention(qx[at:at + m], *kv[s]))
            at += m


def test_calls_on_two_streams_at_once():
    lens, q_lens, hq, hk = [6000, 500], [200, 90], 8, 2
    cache, kv = states(lens, hk, torch.bfloat16, 70)
    work = []
    for i in range(2):
        qd, qx = rand_q(2, hq, torch.bfloat16, 71 + i), rand_q(290, hq, torch.bfloat16, 73 + i)
        work.append((torch.cuda.Stream(), qd, qx, torch.empty_like(qd), torch.empty_like(qx), decode_ws(2, hq, hk, 6000),
                     cross_ws(2, 290, hq, hk, 6000)))
    sl, cu = i32(lens), i32([0, 200, 290])
    torch.cuda.synchronize()
    for _ in range(10):
        for stream, qd, qx, od, ox, ws_d, ws_x in work:
            kvtc.kvtc_raw_decode_attention(cache, 1, qd, sl, 6000, od, ws_d, stream=stream)
            kvtc.kvtc_raw_cross_attention(cache, 1, qx, cu, sl, 6000, ox, ws_x, stream=stream)
    torch.cuda.synchronize()
    assert cache.status.item() == 0
    for _, qd, qx, od, ox, *_ in work:
        for s, (a, b) in enumerate(((0, 200), (200, 290))):
            ref.assert_close(od[s:s + 1], *ref.attention(qd[s:s + 1], *kv[s]))
            ref.assert_close(ox[a:b], *ref.attention(qx[a:b], *kv[s]))


# ------------------------------------------------------------------ step tables
@pytest.mark.parametrize("n_seq,top_new,extra", [(127, 9, 3), (128, 9, 0), (129, 9, 3), (2048, 3, 1), (2049, 3, 1),
                                                 (5000, 2, 0), (100, 700, 5), (1, 5000, 0), (128, 4, 512)])
def test_step_tables_at_the_edges_of_a_block(n_seq, top_new, extra):
    case = tables_case(n_seq + top_new, n_seq, 300, top_new, 48, 4 * n_seq + 3000, extra)
    want = ref.step_tables(*case)
    same_tables(run_tables(*case), want)
    same_tables(run_tables(*case, in_place=True), want)


def test_step_tables_with_one_output_in_place():
    cached, new, ring, state, table, rows = tables_case(3, 3000, 300, 4, 16, 9000, 7)
    want = ref.step_tables(cached, new, ring, state, table, rows)
    for lens_in_place in (False, True):
        c, f, r, st, tb = i32(cached), i32(new), i32(ring), i32(state), i32(table)
        seq = c if lens_in_place else torch.empty_like(c)
        out = torch.empty_like(st) if lens_in_place else st
        cu, pos = torch.empty(3001, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
        slots, ws = torch.empty(rows, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
        kvtc.kvtc_step_tables(c, f, r, st, tb, seq, cu, slots, pos, out, ws)
        torch.cuda.synchronize()
        got = dict(ring=r.cpu().numpy(), state=out.tolist(), table=tb.cpu().numpy(), seq_lens=seq.cpu().numpy(),
                   cu=cu.cpu().numpy(), slots=slots.cpu().numpy(), positions=pos.cpu().numpy())
        for key, val in got.items():
            assert np.array_equal(val, want[key]), key
        assert not ws.any()


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 0), (1, 0, 1), (2, 1024, 5), (9000, 1, 1), (4097, 3, 2)])
def test_rope_of_one_kind_and_of_many_heads(n, hq, hk):
    sections = (20, 4, 40)
    pos = torch.randint(0, 70000, (3, n), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()
    q = rand_q(n, hq, torch.bfloat16, 80) if hq else None
    k = rand_q(n, hk, torch.bfloat16, 81) if hk else None
    qo, ko = (None if x is None else torch.empty_like(x) for x in (q, k))
    kvtc.kvtc_rope(kvtc.rope_desc(sections), q, k, pos, qo, ko)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            ref.assert_close(y, ref.rope(x, pos, sections), ref.rope_bound(x, torch.bfloat16))


def test_rope_and_its_transpose_give_the_rows_back():
    q = torch.randn((300, 6, D), generator=torch.Generator().manual_seed(82)).cuda()
    pos = torch.randint(0, 1 << 30, (300,), generator=torch.Generator().manual_seed(83), dtype=torch.int32).cuda()
    d, out = kvtc.rope_desc([64], base=10000.0), torch.empty_like(q)
    kvtc.kvtc_rope(d, q, None, pos, out, None)
    kvtc.kvtc_rope(d, out, None, pos, out, None, inverse=True)
    # both rotations' errors, the second's on rows as large as the first's
    assert ((out.double() - q.double()).abs() <= 2.5 * ref.rope_bound(q, torch.float32)).all()


# ------------------------------------------------------------------ the binding's refusals
def test_the_binding_refuses_types_shapes_and_strides():
    cache, _ = states([100, 50], 2, torch.bfloat16, 90)
    q, lens = rand_q(2, 4, torch.bfloat16, 91), i32([100, 50])
    out, ws = torch.empty_like(q), decode_ws(2, 4, 2, 100)
    good = dict(q=q, lens=lens, out=out, ws=ws)
    for change, error in ((dict(q=q.half()), TypeError), (dict(lens=lens.long()), TypeError), (dict(out=out.float()), TypeError),
                          (dict(q=q[:1]), ValueError), (dict(q=q[..., :64]), ValueError), (dict(lens=i32([1, 2, 3])), ValueError),
                          (dict(out=out[:, :2]), ValueError), (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                          (dict(lens=lens.cpu()), ValueError), (dict(ws=ws.cpu()), ValueError), (dict(ws=ws[:100]), kvtc.KvtcError)):
        a = dict(good, **change)
        with pytest.raises(error):
            kvtc.kvtc_raw_decode_attention(cache, 1, a["q"], a["lens"], 100, a["out"], a["ws"])
    with pytest.raises(ValueError):                    # beyond the library's int
        kvtc.kvtc_raw_decode_attention(cache, 1, q, lens, 1 << 40, out, ws)
    with pytest.raises(TypeError):
        kvtc.kvtc_raw_decode_attention(cache, "1", q, lens, 100, out, ws)
    with pytest.raises(kvtc.KvtcError):
        kvtc.kvtc_raw_decode_attention(cache, 2, q, lens, 100, out, ws)
    with pytest.raises(kvtc.KvtcError):
        kvtc.kvtc_raw_decode_attention(cache, 1, q, lens, 100, q, ws)
    k = rand_q(3, 2, torch.bfloat16, 92)
    slots = torch.arange(3, device="cuda")
    for bad in (dict(k=rand_q(3, 3, torch.bfloat16, 1)), dict(v=k[:2]), dict(slots=slots[:2]), dict(slots=slots.int()),
                dict(k=k.half()), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1))):
        a = dict(dict(k=k, v=k, slots=slots), **bad)
        with pytest.raises((TypeError, ValueError)):
            kvtc.kvtc_raw_append(cache, 1, a["k"], a["v"], a["slots"])
    with pytest.raises(ValueError):                    # rope without positions
        kvtc.kvtc_raw_append(cache, 1, k, k, slots, rope=kvtc.rope_desc([64]))
    with pytest.raises(ValueError):                    # positions of another shape
        kvtc.kvtc_rope(kvtc.rope_desc([32, 32]), q, None, i32([1, 2]), out, None)
    with pytest.raises(kvtc.KvtcError):                # q without a rotation
        kvtc.kvtc_raw_append(cache, 1, k, k, slots, q=k, q_out=torch.empty_like(k))
    torch.cuda.synchronize()
    assert cache.status.item() == 0


def test_a_stream_handle_an_int_and_the_current_stream():
    cache, kv = states([300], 2, torch.bfloat16, 93)
    q, lens, ws = rand_q(1, 4, torch.bfloat16, 94), i32([300]), decode_ws(1, 4, 2, 300)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        out = torch.full_like(q, float("nan"))
        torch.cuda.synchronize()
        if stream is None:
            with torch.cuda.stream(side):
                kvtc.kvtc_raw_decode_attention(cache, 1, q, lens, 300, out, ws)
        else:
            kvtc.kvtc_raw_decode_attention(cache, 1, q, lens, 300, out, ws, stream=stream)
        side.synchronize()
        ref.assert_close(out, *ref.attention(q, *kv[0]))


@pytest.mark.parametrize("n_seq,rows,max_pages", [(5, (1 << 24) + 3, 16), (130, 40, 1 << 20), (200, 1 << 20, 8)])
def test_step_tables_whose_sums_may_pass_32_bits(n_seq, rows, max_pages):
    # launches padded to very many rows and very wide tables: the scans run in 64 bits
    cached, new, ring, state, table, _ = tables_case(n_seq, n_seq, 300, 3, 16, 2000, 0)
    new[1] = (1 << 31) - 1
    wide = np.full((n_seq, max_pages), -1, np.int32)
    n = min(16, max_pages)
    wide[:, :n] = table[:, :n]
    case = (cached, new, ring, state, wide, rows)
    got, want = run_tables(*case), ref.step_tables(*case)
    assert want["status"] & kvtc.STATUS_BAD_POS
    same_tables(got, want)
