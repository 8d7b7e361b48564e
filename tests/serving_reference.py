"""Plain 64-bit references of the calls around the cache, for the tests."""

import math

import numpy as np
import torch

P, D = 128, 128
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative


def pages(n):
    return (n + P - 1) // P


def step_tables(cached, new, ring, state, table, n_rows):
    """The definition, request by request.  Returns every output and the status bits."""
    ring, table = ring.copy(), table.copy()
    capacity, limit = len(ring), table.shape[1] * P
    head, count = state
    status = 0
    if not (0 <= head < capacity and 0 <= count <= capacity):
        head = count = 0
        status |= 1
    slots, pos = np.full(n_rows, -1, np.int64), np.zeros(n_rows, np.int32)
    seq, cu = [], [0]
    wanted = taken = given = 0
    for s, (c, n) in enumerate(zip(cached, new)):
        bad = c < 0 or c > limit
        if bad:
            status |= 2
            c = 0
        if n < 0:
            for p in range(pages(c)):
                if table[s, p] < 0 or given >= capacity - count:
                    status |= 1
                if given < capacity - count:
                    ring[(head + count + given) % capacity] = table[s, p]
                    given += 1
            seq.append(0)
            cu.append(cu[-1])
            continue
        first = cu[-1]
        cu.append(first + n)
        if bad or c + n > limit or first + n > n_rows:
            if n > 0:
                status |= 2
            seq.append(c)
            continue
        need = pages(c + n) - pages(c)
        wanted += need
        if need and wanted > count:
            status |= 8
            seq.append(c)
            continue
        for p in range(need):
            table[s, pages(c) + p] = ring[(head + taken + p) % capacity]
        taken += need
        seq.append(c + n)
        for i in range(n):
            page = table[s, (c + i) // P]
            if page < 0:
                status |= 1
                continue
            slots[first + i] = int(page) * P + (c + i) % P
            pos[first + i] = c + i
    return dict(ring=ring, state=[(head + taken) % capacity, count - taken + given], table=table,
                seq_lens=np.array(seq, np.int32), cu=np.minimum(cu, n_rows).astype(np.int32), slots=slots,
                positions=pos, status=status)


def pair_axis(sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out, a = list(sections), [], 0
    while len(out) < 64:
        if left[a]:
            left[a] -= 1
            out.append(a)
        a = (a + 1) % len(sections)
    return out


def rope(x, positions, sections, interleaved=False, base=500000.0, inverse=False):
    """x [n][heads][128], positions [n_axes][n], in 64 bits."""
    x, positions = x.double(), positions.reshape(len(sections), -1).double()
    axis = torch.tensor(pair_axis(sections, interleaved), device=x.device)
    f = torch.tensor([math.pow(base, -2.0 * i / D) for i in range(64)], dtype=torch.float64, device=x.device)
    a = (positions[axis].t() * f)[:, None] * (-1.0 if inverse else 1.0)
    lo, hi = x[..., :64], x[..., 64:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def rope_bound(x, dtype, far=1.0):
    """Largest error of a rotated row: the sine and cosine (sincospif within 2 units of fp32,
    its argument rounded once to fp32: 2^-24 * pi at most) and three fp32 roundings, on
    |x_i| + |x_{i+64}|; then the rounding of the result (added by the caller relative to
    it).  Subnormal results of 16-bit types round by half their smallest step."""
    s = x.double().abs()
    s = s[..., :64] + s[..., 64:]
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return torch.cat([s, s], -1) * (12 * 2.0 ** -24) * far + tiny


def attention(q, k, v, scale=1.0 / math.sqrt(D)):
    """q [nq][Hq][128], k, v [n][Hkv][128] -> (o, bound without the output's rounding) in
    64 bits.  The bound: P rounded to the pages' type (u relative, in the sum of p v and in
    the sum of p: 2 u sum p |v|), scores in fp32 (128 products and the scale, the running
    rescale and exp2: (160 * 2^-24) * scale * sum |q k| + 2^-19, each entering p and l)."""
    nq, hq, _ = q.shape
    n, hk, _ = k.shape
    g = hq // hk
    o = torch.zeros((nq, hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    if n == 0:
        return o, bound
    u = U[q.dtype]
    for h in range(hq):
        a, b, c = q[:, h].double(), k[:, h // g].double(), v[:, h // g].double()
        p = torch.softmax(a @ b.t() * scale, -1)
        o[:, h] = p @ c
        spread = (a.abs() @ b.abs().t()).amax(-1, keepdim=True) * scale
        bound[:, h] = (p @ c.abs()) * (2 * u + 2 * (160 * 2.0 ** -24 * spread + 2.0 ** -19))
    return o, bound


def assert_close(got, want, bound):
    """|got - want| <= bound + half a step of the output's type relative to the value."""
    assert torch.isfinite(got).all()
    u = U[got.dtype]
    tol = bound + u * (want.abs() + bound) + 2.0 ** -25
    err = (got.double() - want).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3f} times the bound"


def scatter_states(pool, layer, table, s, k, v):
    """Writes k, v [n][H][128] into the pages of sequence s by plain indexing."""
    t = torch.arange(k.shape[0], device=k.device)
    page = table[s].long()[t // P]
    pool[layer][page, :, 0, t % P] = k.to(pool.dtype)
    pool[layer][page, :, 1, t % P] = v.to(pool.dtype)
