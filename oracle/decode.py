"""Oracle of the decode step's cache, attention and norm operators.

TEST INFRASTRUCTURE, like the rest of this package: plain numpy, no code shared
with the library. Attention and the norm are float64 from the exact input
values; the cache's codes are decided in fp32 with IEEE operations, one value
at a time, as their definition says (so they are compared bit for bit); the
block plan is written as the loop that its definition describes.
"""
from __future__ import annotations

import numpy as np

I8, E4M3 = 0, 1
QMAX = {I8: np.float32(127), E4M3: np.float32(448)}


def _e4m3_table():
    """Values of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa
    bits, exponent 0 subnormal, 0x7F and 0xFF not a number."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c >> 7, -v, v)


E4M3_VALUES = _e4m3_table()


def decode(codes, fmt):
    """uint8 bit patterns -> float64 code values."""
    c = np.asarray(codes, dtype=np.uint8)
    return c.view(np.int8).astype(np.float64) if fmt == I8 else E4M3_VALUES[c]


def encode(x, fmt):
    """fp32 values -> uint8 bit patterns of the nearest codes (ties to even, clamped)."""
    x = np.asarray(x, dtype=np.float32)
    if fmt == I8:
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    a = np.rint(a / step) * step                     # exact: a / step has at most 28 bits
    mags = E4M3_VALUES[:127]
    code = np.searchsorted(mags, a).astype(np.uint8)
    assert np.array_equal(mags[code], a)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def block_plan(old, new, table, free_list, count, bs, max_tokens):
    """The plan one block and one token at a time. Returns (table, free_list,
    count, cu, slots, positions, info)."""
    table, free = np.array(table), np.array(free_list)
    R, maxb = table.shape
    N = len(free)
    ceil = lambda n: -(-int(n) // bs)  # noqa: E731
    none = np.full(max_tokens, -1, np.int32)
    released = [table[r, b] for r in range(R) for b in range(ceil(max(new[r], 0)), ceil(max(old[r], 0)))]
    taken = sum(max(0, ceil(new[r]) - ceil(old[r])) for r in range(R))
    tokens = sum(max(0, int(new[r]) - int(old[r])) for r in range(R))
    state = 0
    if min(old) < 0 or min(new) < 0 or not 0 <= count <= N:
        state = 4
    elif max(max(ceil(n) for n in old), max(ceil(n) for n in new)) > maxb:
        state = 2
    elif count + len(released) > N:
        state = 4
    elif tokens > max_tokens:
        state = 3
    elif taken > count + len(released):
        state = 1
    if state:
        return table, free, count, np.zeros(R + 1, np.int32), none, none.copy(), np.array([0, 0, 0, state], np.int32)
    stack = list(free[:count]) + released[::-1]
    slots, pos, cu, got = none, none.copy(), [0], 0
    for i, b in enumerate(released):
        free[count + len(released) - 1 - i] = b
    for r in range(R):
        for b in range(ceil(old[r]), ceil(new[r])):
            table[r, b] = stack.pop()
        for p in range(int(old[r]), int(new[r])):
            slots[got], pos[got] = table[r, p // bs] * bs + p % bs, p
            got += 1
        cu.append(got)
    return table, free, len(stack), np.array(cu, np.int32), slots, pos, np.array([tokens, taken, len(released), 0],
                                                                                np.int32)


def append(x, slots, cache, scales, fmt, num_blocks, bs):
    """One of the two caches (uint8 patterns [blocks][H][bs][D], scales fp32
    [blocks][H]) after an append of x (fp32 values [T][H][D]); new arrays."""
    cache, scales, x = cache.copy(), scales.copy(), np.asarray(x, np.float32)
    T = len(slots)
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= num_blocks * bs:
            t += 1
            continue
        blk, f = s // bs, s % bs
        n = 1
        while t + n < T and f + n < bs and slots[t + n] == s + n:
            n += 1
        for h in range(cache.shape[1]):
            run = x[t:t + n, h]
            s0 = scales[blk, h] if f else np.float32(0)
            sc = max(s0, np.float32(np.abs(run).max()) / QMAX[fmt])
            if f and sc > s0:
                ratio = np.float32(s0) / np.float32(sc)
                cache[blk, h, :f] = encode(decode(cache[blk, h, :f], fmt).astype(np.float32) * ratio, fmt)
            cache[blk, h, f:f + n] = encode(run / sc if sc > 0 else np.zeros_like(run), fmt)
            if f == 0:
                cache[blk, h, n:] = 0
            scales[blk, h] = sc
        t += n
    return cache, scales


def attention(q, k_cache, v_cache, scales, table, ctx_lens, cu_q, fmt, softmax_scale, tree=None):
    """float64 attention of q [T][Hq][D] over uint8-pattern caches. Returns
    five arrays: out [T][Hq][D]; sum p |v| [T][Hq][D]; and [T][Hq] each: the
    largest sum |q_d k_d| * softmax_scale of a seen token, the number of seen
    tokens, the largest |v|."""
    T, Hq, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    G = Hq // Hkv
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    qk, seen_n, vmax = np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for r in range(len(ctx_lens)):
        ctx = min(int(ctx_lens[r]), table.shape[1] * bs)
        n = int(cu_q[r + 1] - cu_q[r])
        if n == 0 or ctx <= 0:
            continue
        tok = np.arange(ctx)
        blk = table[r, tok // bs].astype(np.int64)
        good = (blk >= 0) & (blk < nb)
        safe = np.where(good, blk, 0)
        for h in range(Hkv):
            K = decode(k_cache[safe, h, tok % bs], fmt) * scales[safe, h, 0].astype(np.float64)[:, None]
            V = decode(v_cache[safe, h, tok % bs], fmt) * scales[safe, h, 1].astype(np.float64)[:, None]
            for i in range(n):
                t = int(cu_q[r]) + i
                base = ctx - n
                if tree is not None and n <= 32:
                    bits = (int(tree[t]) >> np.clip(tok - base, 0, 31)) & 1
                    see = good & ((tok < base) | (bits == 1))
                else:
                    see = good & (tok <= base + i)
                if not see.any():
                    continue
                Ks, Vs = K[see], V[see]
                for hq in range(h * G, (h + 1) * G):
                    qq = q[t, hq].astype(np.float64)
                    s = Ks @ qq * softmax_scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, hq], mag[t, hq] = p @ Vs, p @ np.abs(Vs)
                    qk[t, hq] = (np.abs(Ks) @ np.abs(qq)).max() * softmax_scale
                    seen_n[t, hq], vmax[t, hq] = see.sum(), np.abs(Vs).max()
    return out, mag, qk, seen_n, vmax


def attention_shared(q, k_cache, v_cache, scales, ptable, plens, cu_req, table, ctx_lens, cu_q, fmt, softmax_scale,
                     tree=None):
    """As attention, for requests that see the tokens of their group's prefix
    (ptable, plens; group g has the requests cu_req[g] .. cu_req[g + 1] - 1) before
    their own."""
    T, Hq, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    G = Hq // Hkv
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    qk, seen_n, vmax = np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    group_of = {r: g for g in range(len(plens)) for r in range(int(cu_req[g]), int(cu_req[g + 1]))}

    def tokens(row, n):
        tok = np.arange(n)
        blk = row[tok // bs].astype(np.int64)
        return np.where((blk >= 0) & (blk < nb), blk, -1), tok % bs

    for r in range(len(ctx_lens)):
        n = int(cu_q[r + 1] - cu_q[r])
        ctx = min(max(int(ctx_lens[r]), 0), table.shape[1] * bs)
        pre = min(max(int(plens[group_of[r]]), 0), ptable.shape[1] * bs) if r in group_of else 0
        blk, slot = tokens(table[r], ctx)
        if pre:
            pb, ps = tokens(ptable[group_of[r]], pre)
            blk, slot = np.concatenate((pb, blk)), np.concatenate((ps, slot))
        good, safe = blk >= 0, np.where(blk >= 0, blk, 0)
        tok, base = np.arange(pre + ctx), pre + ctx - n
        if n == 0 or pre + ctx == 0:
            continue
        see = np.zeros((n, pre + ctx), bool)
        for i in range(n):
            if tree is not None and n <= 32:
                bits = (int(tree[int(cu_q[r]) + i]) >> np.clip(tok - base, 0, 31)) & 1
                see[i] = good & ((tok < base) | (tok < pre) | (bits == 1))
            else:
                see[i] = good & ((tok <= base + i) | (tok < pre))
        live = see.any(1)
        at = int(cu_q[r]) + np.arange(n)[live]
        if not live.any():
            continue
        for h in range(Hkv):
            K = decode(k_cache[safe, h, slot], fmt) * scales[safe, h, 0].astype(np.float64)[:, None]
            V = decode(v_cache[safe, h, slot], fmt) * scales[safe, h, 1].astype(np.float64)[:, None]
            used = see.any(0)
            V = np.where(used[:, None], V, 0.0)
            for hq in range(h * G, (h + 1) * G):
                qq = q[at, hq].astype(np.float64)
                s = np.where(see[live], qq @ K.T * softmax_scale, -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[at, hq], mag[at, hq] = p @ V, p @ np.abs(V)
                qk[at, hq] = np.where(see[live], np.abs(qq) @ np.abs(K).T, 0).max(1) * softmax_scale
                seen_n[at, hq] = see[live].sum(1)
                vmax[at, hq] = np.where(see[live], np.abs(V).max(1), 0).max(1)
    return out, mag, qk, seen_n, vmax


def rmsnorm(h, weight, eps, sign_bits=None):
    """float64 y (or its randomized Hadamard transform) of the stored rows h;
    also sum |y| of each value's 32-block (or |y| itself)."""
    h = np.asarray(h, np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if sign_bits is None:
        return y, np.abs(y)
    M, K = y.shape
    bits = (np.asarray(sign_bits).view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    z = y.reshape(M, K // 32, 32) * (1.0 - 2.0 * bits)
    i = np.arange(32)
    H = np.array([[(-1.0) ** bin(a & b).count("1") for b in i] for a in i])
    mag = np.broadcast_to(np.abs(z).sum(-1, keepdims=True), z.shape)
    return (z @ H).reshape(M, K), mag.reshape(M, K)


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of the sampler in float64: (order: the tokens above -infinity as
    they rank, C: their summed weights, kept: how many stay, place: of the drawn
    one in the order). x fp32 or bf16 values, finite largest number 3.4e38."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(np.asarray(x, np.float64), np.float64(np.finfo(np.float32).max)))
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if len(order) == 0:
        return order, np.zeros(0), 0, -1
    d = x[order] - x[order[0]]
    if not temperature > 0:
        return order, np.ones(len(order)), 1, 0
    C = np.cumsum(np.exp(d / min(float(temperature), 1e30)))
    n = len(order) if not 0 < top_k < len(x) else min(int(top_k), len(order))
    if top_p < 1:
        n = min(n, int((C[:n] < float(top_p) * C[n - 1]).sum()) + 1)
    if min_p > 0:
        n = min(n, int((d >= float(temperature) * np.log(min(1.0, float(min_p)))).sum()))
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    return order, C, n, min(int((C[:n] <= u * C[n - 1]).sum()), n - 1)
