"""Cases of the serving operators around the cache, with their plain torch forms.

A case is a dict of plain values.  ``prepare`` makes what a program has in hand before
the call, ``run`` makes one pass (the plain form, or the library's calls where ``own`` is
true), ``exact`` computes the definition in 64 bits and ``work`` counts the bytes and
operations that the pass cannot do without.

Operators:

* ``tables``: block tables, slot map, positions and lengths of one serving step from the
  request lengths, pages taken from and given back to a ring of free pages.
* ``rope``: rotary positions with several axes on q and k, forward or transposed.
* ``append``: K and V rows written into uncompressed pages by slot, the rotation of k
  (and of q) in the same pass.
* ``decode``: attention of one new token per sequence over uncompressed pages.
* ``cross``: attention of ragged queries to an encoder's states held in such pages.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 128   # tokens of a page
DIM = 128    # head dimension
BASE = 500000.0
BAD_PAGE, BAD_POS, NO_PAGE = 1, 2, 8
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 16 requests of up to 32k tokens, one new token each: the
        # tables of the smallest serving step, where only latency counts
        dict(name="tables_decode_16", op="tables", n_seq=16, cached=32768, new=1, rows=16, retire=1),
        # an admission step: 2048 requests, most of them with a ragged chunk of prompt,
        # some finishing, rows padded to a fixed launch size
        dict(name="tables_chunks_2048", op="tables", n_seq=2048, cached=8192, new=512, rows=600000, retire=97),
        # q and k of a video-and-text prompt, three position axes, fp32 model, an odd
        # token count, 7 query heads per KV head; transposed (the gradient of q and k)
        dict(name="rope_f32_4097_transposed", op="rope", tokens=4097, q_heads=28, kv_heads=4, dtype="f32",
             sections="16,24,24", interleaved=False, inverse=True),
        # q and k of a long prompt before the coded cache takes them: one axis, bf16,
        # heads as slices of one fused projection
        dict(name="rope_bf16_32768", op="rope", tokens=32768, q_heads=32, kv_heads=8, dtype="bf16",
             sections="64", interleaved=False, inverse=False),
        # one decode step's write: 16 tokens, k and q rotated in the same pass
        dict(name="append_step_16", op="append", tokens=16, q_heads=32, kv_heads=8, dtype="bf16",
             sections="24,20,20", interleaved=True, rotate=True, skip=0),
        # a batch of prompts written at once, three axes, with padding rows in it
        dict(name="append_prompts_16411", op="append", tokens=16411, q_heads=32, kv_heads=8, dtype="bf16",
             sections="16,24,24", interleaved=False, rotate=True, skip=37),
        # a small batch of short chats, one of them empty: latency
        dict(name="decode_short_f16", op="decode", lens="1000,0,517", q_heads=32, kv_heads=8, dtype="f16"),
        # one long document, 7 query heads per KV head: the split over the length
        dict(name="decode_one_131072", op="decode", lens="131072", q_heads=28, kv_heads=4, dtype="bf16"),
        # the 16 x 32k batch that the coded cache's sweep uses
        dict(name="decode_16x32768", op="decode", lens=",".join(["32768"] * 16), q_heads=32, kv_heads=8, dtype="bf16"),
        # the first tokens of a few answers over an encoder's states
        dict(name="cross_first_tokens_f16", op="cross", q_lens="4,1,17", lens="1501,700,1500", q_heads=20,
             kv_heads=20, dtype="f16"),
        # a batch of transcripts scored at once, ragged on both sides, one without states
        dict(name="cross_ragged_8", op="cross", q_lens="448,391,5,448,200,448,63,130",
             lens="1500,1500,1103,0,1500,997,1500,128", q_heads=32, kv_heads=8, dtype="bf16"),
        # a long answer over a long document's states: bound by the matrix products
        dict(name="cross_16384x16384", op="cross", q_lens="16384", lens="16384", q_heads=32, kv_heads=8,
             dtype="bf16"),
    ]


def _text(numbers):
    return ",".join(str(n) for n in numbers)


def _ints(text):
    return [int(n) for n in text.split(",")]


def _row_lens(case):
    """Query rows and states of each sequence of an attention case."""
    lens = _ints(case["lens"])
    return (_ints(case["q_lens"]) if case["op"] == "cross" else [1] * len(lens)), lens


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    while kv * group > 64:
        group = rng.choice([1, 2, 3, 4])
    return kv * group, kv


def _sections(rng):
    n_axes = rng.randint(1, 4)
    cuts = sorted(rng.randint(1, 63) for _ in range(n_axes - 1))
    edges = [0] + cuts + [64]
    return _text(b - a for a, b in zip(edges, edges[1:])), bool(rng.getrandbits(1))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "decode", "cross"])
    if op == "tables":
        n_seq = _log_int(rng, 1, 2048)
        new = rng.choice([1, 1, _log_int(rng, 1, max(1, min(8192, 524288 // n_seq)))])
        return dict(op=op, n_seq=n_seq, cached=_log_int(rng, 1, 16384), new=new,
                    rows=n_seq * new + rng.choice([0, 0, rng.randint(1, 1000)]), retire=rng.randint(0, n_seq // 3))
    if op in ("rope", "append"):
        q_heads, kv_heads = _heads(rng)
        sections, inter = _sections(rng)
        most = max(1, 1200000 // (q_heads + 2 * kv_heads))
        case = dict(op=op, tokens=_log_int(rng, 1, min(32768, most)), q_heads=q_heads, kv_heads=kv_heads,
                    sections=sections, interleaved=inter)
        if op == "rope":
            return dict(case, dtype=rng.choice(["bf16", "f16", "f32"] if case["tokens"] <= 16384 else ["bf16", "f16"]),
                        inverse=bool(rng.getrandbits(1)))
        return dict(case, dtype=rng.choice(["bf16", "f16"]), rotate=rng.random() < 0.75,
                    skip=rng.choice([0, rng.randint(0, max(0, case["tokens"] // 3))]))
    q_heads, kv_heads = _heads(rng)
    dtype = rng.choice(["bf16", "f16"])
    if op == "decode":
        n_seq = _log_int(rng, 1, 128)
        most = max(1, min(131072, 4000000 // (n_seq * kv_heads)))
        top = _log_int(rng, 1, most)
        lens = [0 if rng.random() < 0.05 else _log_int(rng, 1, top) for _ in range(n_seq)]
        return dict(op=op, lens=_text(lens), q_heads=q_heads, kv_heads=kv_heads, dtype=dtype)
    n_seq = _log_int(rng, 1, 16)
    top_q = _log_int(rng, 1, max(1, 8192 // n_seq))
    top_k = _log_int(rng, 1, 16384 // n_seq)
    q_lens = [0 if rng.random() < 0.05 else rng.randint(1, top_q) for _ in range(n_seq)]
    if sum(q_lens) == 0:
        q_lens[0] = 1
    lens = [0 if rng.random() < 0.05 else rng.randint(1, top_k) for _ in range(n_seq)]
    return dict(op=op, q_lens=_text(q_lens), lens=_text(lens), q_heads=q_heads, kv_heads=kv_heads, dtype=dtype)


# ------------------------------------------------------------------------------ inputs
def _pages(n):
    return (n + PAGE - 1) // PAGE


def _table_lens(case):
    """Cached and new lengths of a tables case (their order is the seed's)."""
    r = random.Random("%d %d %d %d" % (case["n_seq"], case["cached"], case["new"], case["retire"]))
    n = case["n_seq"]
    cached = [0 if r.random() < 0.1 else r.randint(1, case["cached"]) for _ in range(n)]
    if case["new"] == 1:
        new = [1] * n
    else:
        new = [1 if r.random() < 0.25 else r.randint(0, case["new"]) for _ in range(n)]
    for s in r.sample(range(n), case["retire"]):
        new[s] = -1
    return cached, new


def _random(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _positions(case, tokens, gen):
    """Positions as a prompt with images has them: the axes run apart inside an image."""
    base = torch.arange(tokens, device="cuda", dtype=torch.int64)
    start = int(torch.randint(0, 100000, (1,), generator=gen, device="cuda").item())
    rows = [start + base]
    for a in range(1, len(_ints(case["sections"]))):
        jump = torch.randint(0, 64, (tokens,), generator=gen, device="cuda")
        rows.append(start + base + jump * a)
    return torch.stack(rows).to(torch.int32).contiguous()


def _prepare_tables(case, seed):
    r = random.Random(seed)
    cached, new = _table_lens(case)
    order = list(range(case["n_seq"]))
    r.shuffle(order)
    cached = [cached[i] for i in order]
    new = [new[i] for i in order]
    max_pages = _pages(case["cached"] + max(1, case["new"]))
    held = [_pages(c) for c in cached]
    need = sum(_pages(c + n) - _pages(c) for c, n in zip(cached, new) if n >= 0)
    spare = 5 + need // 7
    capacity = sum(held) + need + spare
    ids = np.random.default_rng(seed).permutation(capacity).astype(np.int32)
    table = np.full((case["n_seq"], max_pages), -1, np.int32)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        at += h
    free = need + spare
    head = r.randrange(capacity)
    ring = np.full(capacity, -1, np.int32)
    ring[(head + np.arange(free)) % capacity] = ids[at:]

    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    n_seq, rows = case["n_seq"], case["rows"]
    return dict(case=case, cached=dev(np.array(cached, np.int32)), new=dev(np.array(new, np.int32)), ring=dev(ring),
                ring_state=dev(np.array([head, free], np.int32)), table=dev(table),
                seq_lens=torch.empty(n_seq, dtype=torch.int32, device="cuda"),
                cu=torch.empty(n_seq + 1, dtype=torch.int32, device="cuda"),
                slots=torch.empty(rows, dtype=torch.int64, device="cuda"),
                positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                ring_out=torch.empty(2, dtype=torch.int32, device="cuda"),
                workspace=torch.zeros(4, dtype=torch.int32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _qkv(case, gen):
    """q, k and v as the slices of one fused projection's output."""
    t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
    x = _random((t, hq + 2 * hk, DIM), DTYPES[case["dtype"]], gen)
    return x, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def _prepare_rope(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, q, k, _ = _qkv(case, gen)
    state = dict(case=case, x=x, q=q, k=k, positions=_positions(case, case["tokens"], gen),
                 q_out=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
                 k_out=torch.empty(k.shape, dtype=k.dtype, device="cuda"))
    if own:
        from bit_quantization_head_b200 import kvtc
        state["desc"] = kvtc.rope_desc(_ints(case["sections"]), case["interleaved"], BASE)
    return state


def _prepare_append(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, q, k, v = _qkv(case, gen)
    t = case["tokens"]
    n_pages = _pages(t) + 3
    # the tokens' slots: pages in shuffled order, a prompt's tokens in a row, some rows padding
    order = np.random.default_rng(seed).permutation(n_pages)
    at = np.arange(t) + seed % PAGE
    slots = order[at // PAGE].astype(np.int64) * PAGE + at % PAGE
    if case["skip"]:
        slots[-case["skip"]:] = -1
    state = dict(case=case, x=x, q=q, k=k, v=v, positions=_positions(case, t, gen), slots=torch.from_numpy(slots).cuda(),
                 pool=_random((2, n_pages, case["kv_heads"], 2, PAGE, DIM), k.dtype, gen),
                 q_out=torch.empty(q.shape, dtype=q.dtype, device="cuda"))
    if own:
        from bit_quantization_head_b200 import kvtc
        state["desc"] = kvtc.rope_desc(_ints(case["sections"]), case["interleaved"], BASE)
        state["cache"] = kvtc.RawCache(2, case["kv_heads"], n_pages, torch.zeros((1, 1), dtype=torch.int32),
                                       dtype=k.dtype, pool=state["pool"])
    return state


def _prepare_attention(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q_lens, lens = _row_lens(case)
    hq, hk, dtype = case["q_heads"], case["kv_heads"], DTYPES[case["dtype"]]
    n_seq = len(lens)
    max_pages = max(1, max(_pages(n) for n in lens))
    used = sum(_pages(n) for n in lens)
    n_pages = used + 2
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table = np.full((n_seq, max_pages), -1, np.int32)
    pool = torch.empty((2, n_pages, hk, 2, PAGE, DIM), dtype=dtype, device="cuda")
    pool[0] = float("nan")  # another layer's pages
    for p in range(0, n_pages, 512):
        pool[1, p:p + 512] = _random(pool[1, p:p + 512].shape, dtype, gen)
    at = 0
    for s, n in enumerate(lens):
        table[s, :_pages(n)] = ids[at:at + _pages(n)]
        at += _pages(n)
        if n % PAGE:  # slots no token has been written to hold anything
            pool[1, int(ids[at - 1]), :, :, n % PAGE:] = float("nan")
    table = torch.from_numpy(table).cuda()
    # some query heads attend sharply, some flatly
    sharp = torch.linspace(0.5, 3.0, hq, device="cuda").view(1, hq, 1)
    rows = sum(q_lens)
    q = (torch.randn((rows, hq, DIM), generator=gen, device="cuda") * sharp).to(dtype)
    state = dict(case=case, pool=pool, table=table, q=q, max_len=max(lens),
                 seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 out=torch.empty((rows, hq, DIM), dtype=dtype, device="cuda"))
    if case["op"] == "cross":
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        state["cu_q"] = torch.from_numpy(cu).cuda()
    if own:
        from bit_quantization_head_b200 import kvtc
        state["cache"] = kvtc.RawCache(2, hk, n_pages, table, dtype=dtype, pool=pool)
        if case["op"] == "decode":
            size = kvtc.kvtc_raw_decode_workspace_bytes(n_seq, hq, hk, state["max_len"])
        else:
            size = kvtc.kvtc_raw_cross_workspace_bytes(n_seq, rows, hq, hk, state["max_len"])
        state["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return state


def prepare(case, seed):
    if case["op"] == "tables":
        return _prepare_tables(case, seed)
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    if case["op"] == "append":
        return _prepare_append(case, seed)
    return _prepare_attention(case, seed)


# ------------------------------------------------------------------------------ plain forms
def _plain_tables(st):
    table, ring = st["table"], st["ring"]
    n_seq, max_pages = table.shape
    rows, capacity = st["slots"].numel(), ring.numel()
    c, n = st["cached"].long(), st["new"].long()
    head, count = st["ring_state"][0].long(), st["ring_state"][1].long()
    retired = n < 0
    fresh = n.clamp(min=0)
    cu = torch.cumsum(fresh, 0)
    held = (c + PAGE - 1) // PAGE
    fits = ~retired & (c + fresh <= max_pages * PAGE) & (cu <= rows)
    need = torch.where(fits, (c + fresh + PAGE - 1) // PAGE - held, torch.zeros_like(c))
    end = torch.cumsum(need, 0)
    grows = fits & ((need == 0) | (end <= count))
    first = end - need
    taken = torch.where(grows, end, torch.zeros_like(end)).amax()
    released = torch.where(retired, held, torch.zeros_like(held))
    rel_first = torch.cumsum(released, 0) - released
    page = torch.arange(max_pages, device="cuda").view(1, -1)
    # the pages of retired sequences go to the ring's tail
    at = (head + count + rel_first.view(-1, 1) + page) % capacity
    at = torch.where(retired.view(-1, 1) & (page < held.view(-1, 1)), at, torch.full_like(at, capacity))
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer.index_put_((at.view(-1),), table.reshape(-1))
    # the new pages come from its head
    take = (head + first.view(-1, 1) + page - held.view(-1, 1)) % capacity
    new_page = grows.view(-1, 1) & (page >= held.view(-1, 1)) & (page < (held + need).view(-1, 1))
    table.copy_(torch.where(new_page, ring[take], table))
    ring.copy_(longer[:capacity])
    st["seq_lens"].copy_(torch.where(retired, torch.zeros_like(c), torch.where(grows, c + fresh, c)))
    st["cu"][:1].zero_()
    st["cu"][1:].copy_(cu.clamp(max=rows))
    st["ring_out"].copy_(torch.stack([(head + taken) % capacity, count - taken + released.sum()]))
    t = torch.arange(rows, device="cuda")
    s = torch.searchsorted(cu, t, right=True)
    inside = s < n_seq
    s = s.clamp(max=n_seq - 1)
    pos = c[s] + t - (cu[s] - fresh[s])
    live = inside & grows[s]
    pos = torch.where(live, pos, torch.zeros_like(pos))
    pid = table[s, pos // PAGE].long()
    st["slots"].copy_(torch.where(live, pid * PAGE + pos % PAGE, torch.full_like(pos, -1)))
    st["positions"].copy_(pos)
    return dict(block_table=table, page_ring=ring, ring_state=st["ring_out"], seq_lens=st["seq_lens"],
                cu_seqlens=st["cu"], slot_map=st["slots"], positions=st["positions"])


def _axis_of_pair(case):
    """The position axis of each of the 64 rotated pairs."""
    sections = _ints(case["sections"])
    if not case["interleaved"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, axis, a = list(sections), [], 0
    while len(axis) < DIM // 2:
        if left[a]:
            left[a] -= 1
            axis.append(a)
        a = (a + 1) % len(sections)
    return axis


def _cos_sin(case, positions, dtype):
    axis = torch.tensor(_axis_of_pair(case), device="cuda")
    freq = BASE ** (-2.0 * torch.arange(DIM // 2, device="cuda", dtype=torch.float64) / DIM)
    angle = positions[axis].double().t() * freq  # [tokens][64]: far positions need 64 bits
    sign = -1.0 if case.get("inverse") else 1.0
    return torch.cos(angle).to(dtype).unsqueeze(1), (sign * torch.sin(angle)).to(dtype).unsqueeze(1)


def _rotate(x, cos, sin):
    a, b = x[..., :DIM // 2].to(cos.dtype), x[..., DIM // 2:].to(cos.dtype)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_rope(st):
    cos, sin = _cos_sin(st["case"], st["positions"], torch.float32)
    return dict(q=_rotate(st["q"], cos, sin).to(st["q"].dtype), k=_rotate(st["k"], cos, sin).to(st["k"].dtype))


def _plain_append(st):
    case, pool = st["case"], st["pool"]
    q, k = st["q"], st["k"]
    if case["rotate"]:
        cos, sin = _cos_sin(case, st["positions"], torch.float32)
        q, k = _rotate(q, cos, sin).to(q.dtype), _rotate(k, cos, sin).to(k.dtype)
    slots = st["slots"][:case["tokens"] - case["skip"]]
    page, row = slots // PAGE, slots % PAGE
    pool[1][page, :, 0, row] = k[:slots.numel()]
    pool[1][page, :, 1, row] = st["v"][:slots.numel()]
    return dict(q=q, pool=pool) if case["rotate"] else dict(pool=pool)


def _softmax_rows(s):
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _states(st, s, dtype):
    """K and V of sequence s, [kv_heads][len][128], gathered from its pages."""
    n = _row_lens(st["case"])[1][s]
    x = st["pool"][1][st["table"][s, :_pages(n)].long()].to(dtype)    # [pages][heads][2][128][128]
    x = x.permute(2, 1, 0, 3, 4).reshape(2, st["case"]["kv_heads"], -1, DIM)[:, :, :n]
    return x[0], x[1]


def _attend(st, dtype):
    """Softmax attention of every query row over its sequence's states, in ``dtype``."""
    case = st["case"]
    hq, hk = case["q_heads"], case["kv_heads"]
    g = hq // hk
    out = torch.zeros(st["q"].shape, dtype=dtype, device="cuda")
    q_lens, lens = _row_lens(case)
    row = 0
    for s, (nq, n) in enumerate(zip(q_lens, lens)):
        if nq and n:
            k, v = _states(st, s, dtype)
            q = st["q"][row:row + nq].to(dtype).view(nq, hk, g, DIM).permute(1, 2, 0, 3).reshape(hk, g * nq, DIM)
            step = max(1, (1 << 28) // n)  # query rows whose scores are held at once
            heads = max(1, step // (g * nq))
            for h in range(0, hk, heads):
                for i in range(0, g * nq, step):
                    scores = q[h:h + heads, i:i + step] @ k[h:h + heads].transpose(1, 2) * (1.0 / math.sqrt(DIM))
                    q[h:h + heads, i:i + step] = _softmax_rows(scores) @ v[h:h + heads]
            out[row:row + nq] = q.view(hk, g, nq, DIM).permute(2, 0, 1, 3).reshape(nq, hq, DIM)
        row += nq
    return out


def _plain_attention(st):
    return _attend(st, torch.float32).to(st["q"].dtype)


# ------------------------------------------------------------------------------ the library's calls
def _own(st):
    from bit_quantization_head_b200 import kvtc
    case = st["case"]
    if case["op"] == "tables":
        kvtc.kvtc_step_tables(st["cached"], st["new"], st["ring"], st["ring_state"], st["table"], st["seq_lens"],
                              st["cu"], st["slots"], st["positions"], st["ring_out"], st["workspace"], st["status"])
        return dict(block_table=st["table"], page_ring=st["ring"], ring_state=st["ring_out"],
                    seq_lens=st["seq_lens"], cu_seqlens=st["cu"], slot_map=st["slots"], positions=st["positions"])
    if case["op"] == "rope":
        kvtc.kvtc_rope(st["desc"], st["q"], st["k"], st["positions"], st["q_out"], st["k_out"],
                       inverse=case["inverse"])
        return dict(q=st["q_out"], k=st["k_out"])
    if case["op"] == "append":
        if case["rotate"]:
            kvtc.kvtc_raw_append(st["cache"], 1, st["k"], st["v"], st["slots"], rope=st["desc"],
                                 positions=st["positions"], q=st["q"], q_out=st["q_out"])
            return dict(q=st["q_out"], pool=st["pool"])
        kvtc.kvtc_raw_append(st["cache"], 1, st["k"], st["v"], st["slots"])
        return dict(pool=st["pool"])
    if case["op"] == "decode":
        kvtc.kvtc_raw_decode_attention(st["cache"], 1, st["q"], st["seq_lens"], st["max_len"], st["out"],
                                       st["workspace"])
    else:
        kvtc.kvtc_raw_cross_attention(st["cache"], 1, st["q"], st["cu_q"], st["seq_lens"], st["max_len"], st["out"],
                                      st["workspace"])
    return st["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tables":
        return _plain_tables(state)
    if op == "rope":
        return _plain_rope(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ------------------------------------------------------------------------------ the definition in 64 bits
def _exact_tables(st):
    """Request by request on the host, as the definition reads."""
    cached, new = st["cached"].tolist(), st["new"].tolist()
    ring, table = st["ring"].cpu().numpy().copy(), st["table"].cpu().numpy().copy()
    head, count = st["ring_state"].tolist()
    capacity, rows, limit = len(ring), st["slots"].numel(), table.shape[1] * PAGE
    slots, positions = np.full(rows, -1, np.int64), np.zeros(rows, np.int32)
    seq_lens, cu = [], [0]
    wanted = taken = given = 0
    for s, (c, n) in enumerate(zip(cached, new)):
        if n < 0:
            for p in range(_pages(c)):
                ring[(head + count + given) % capacity] = table[s, p]
                given += 1
            seq_lens.append(0)
            cu.append(cu[-1])
            continue
        first, last = cu[-1], cu[-1] + n
        cu.append(last)
        if c + n > limit or last > rows:
            seq_lens.append(c)
            continue
        need = _pages(c + n) - _pages(c)
        wanted += need
        if need and wanted > count:
            seq_lens.append(c)
            continue
        for p in range(need):
            table[s, _pages(c) + p] = ring[(head + taken + p) % capacity]
        taken += need
        seq_lens.append(c + n)
        pos = np.arange(c, c + n)
        positions[first:last] = pos
        slots[first:last] = table[s, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE

    def dev(x, dtype):
        return torch.from_numpy(np.ascontiguousarray(x, dtype)).cuda()

    return dict(block_table=dev(table, np.int32), page_ring=dev(ring, np.int32),
                ring_state=dev([(head + taken) % capacity, count - taken + given], np.int32),
                seq_lens=dev(seq_lens, np.int32), cu_seqlens=dev(np.minimum(cu, rows), np.int32),
                slot_map=dev(slots, np.int64), positions=dev(positions, np.int32))


def _exact_rotate(case, x, positions):
    """Each pair as a complex number times e^{ia}, in 64 bits."""
    pos = positions.double()
    turn = torch.empty((x.shape[0], DIM // 2), dtype=torch.float64, device="cuda")
    for i, a in enumerate(_axis_of_pair(case)):
        turn[:, i] = pos[a] * math.pow(BASE, -i / 64.0)
    if case.get("inverse"):
        turn = -turn
    z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * torch.polar(torch.ones_like(turn), turn)[:, None]
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_attention(st):
    """Sequence by sequence and head by head; the softmax through its log-sum-exp."""
    case = st["case"]
    hq, hk = case["q_heads"], case["kv_heads"]
    q_lens, lens = _row_lens(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for s, (nq, n) in enumerate(zip(q_lens, lens)):
        pages = st["table"][s, :_pages(n)].long()
        for h in range(hk if nq and n else 0):
            k = st["pool"][1, pages, h, 0].reshape(-1, DIM)[:n].double()
            v = st["pool"][1, pages, h, 1].reshape(-1, DIM)[:n].double()
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                for i in range(row, row + nq, 8192):
                    e = min(i + 8192, row + nq)
                    x = torch.mm(st["q"][i:e, j].double(), k.t()).div_(math.sqrt(DIM))
                    x.sub_(torch.logsumexp(x, dim=1, keepdim=True)).exp_()
                    out[i:e, j] = torch.mm(x, v)
        row += nq
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(st)
    if case["op"] == "rope":
        return dict(q=_exact_rotate(case, st["q"], st["positions"]), k=_exact_rotate(case, st["k"], st["positions"]))
    if case["op"] == "append":
        pool = st["pool"].double()
        k = _exact_rotate(case, st["k"], st["positions"]) if case["rotate"] else st["k"].double()
        slots = st["slots"][st["slots"] >= 0]
        flat = pool[1].permute(0, 3, 1, 2, 4).reshape(-1, case["kv_heads"], 2, DIM)   # by slot
        flat[slots] = torch.stack([k, st["v"].double()], dim=2)[:slots.numel()]
        pool[1] = flat.view(pool.shape[1], PAGE, case["kv_heads"], 2, DIM).permute(0, 2, 3, 1, 4)
        if not case["rotate"]:
            return dict(pool=pool)
        return dict(q=_exact_rotate(case, st["q"], st["positions"]), pool=pool)
    return _exact_attention(st)


# ------------------------------------------------------------------------------ work
def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}.get(case.get("dtype"), 4)
    if case["op"] == "tables":
        cached, new = _table_lens(case)
        # pages that tokens are mapped to are read (from the table or the ring), new ones
        # and returned ones written; 12 bytes per row
        touched = sum(_pages(c + n) - c // PAGE for c, n in zip(cached, new) if n > 0)
        moved = sum(_pages(c + n) - _pages(c) if n >= 0 else 2 * _pages(c) for c, n in zip(cached, new))
        return {"bytes": 16 * case["n_seq"] + 4 * (touched + moved) + 12 * case["rows"] + 20, "flops": 0}
    if case["op"] in ("rope", "append"):
        t, hq, hk, axes = case["tokens"], case["q_heads"], case["kv_heads"], len(_ints(case["sections"]))
        if case["op"] == "rope":
            return {"bytes": 2 * t * (hq + hk) * DIM * size + 4 * axes * t, "flops": 3 * t * (hq + hk) * DIM}
        kept = t - case["skip"]
        moved, turned = 4 * kept * hk * DIM * size + 8 * t, 0
        if case["rotate"]:
            moved += 2 * t * hq * DIM * size + 4 * axes * t
            turned = 3 * DIM * (t * hq + kept * hk)
        return {"bytes": moved, "flops": turned}
    hq, hk = case["q_heads"], case["kv_heads"]
    q_lens, lens = _row_lens(case)
    rows = sum(q_lens)
    states = sum(n for nq, n in zip(q_lens, lens) if nq)
    pairs = sum(nq * n for nq, n in zip(q_lens, lens))
    return {"bytes": 2 * rows * hq * DIM * size + 2 * states * hk * DIM * size + 4 * (states // PAGE + 2 * len(q_lens)),
            "flops": 4 * DIM * hq * pairs}
