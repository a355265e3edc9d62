"""Workloads of the decode step around the quantized products: the paged 8-bit
key/value cache (block plan, append, attention) and the residual RMS norm.

`listed()` gives named cases, `draw()` further ones of the same ranges,
`prepare()` the inputs of a case on the GPU, `run()` one pass through the
operator: with `own` false in plain torch operations, with `own` true through
the library's entry points. `exact()` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = {"i8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one chat turn's first tokens: a context shorter than three pages, all latency
        dict(name="attn_short", op="attn", R=1, q=1, ctx=37, ragged=False, tree=False, Hq=32, Hkv=8, D=128, bs=16,
             fmt="i8"),
        # batch-one decode of the 9B-class layer (32 query and 8 key/value heads of 128) far into a long document
        dict(name="attn_long", op="attn", R=1, q=1, ctx=131071, ragged=False, tree=False, Hq=32, Hkv=8, D=128, bs=64,
             fmt="i8"),
        # continuous batching: 32 requests, each one token, contexts from one token to 8192
        dict(name="attn_batch", op="attn", R=32, q=1, ctx=8192, ragged=True, tree=False, Hq=32, Hkv=8, D=128, bs=16,
             fmt="e4m3"),
        # speculative-tree verification: 16 draft tokens under a tree mask over a long context
        dict(name="attn_tree", op="attn", R=1, q=16, ctx=32784, ragged=False, tree=True, Hq=32, Hkv=8, D=128, bs=64,
             fmt="i8"),
        # a small model's batch of requests with five draft tokens each (a chain, no tree), heads of 64
        dict(name="attn_draft", op="attn", R=6, q=5, ctx=5000, ragged=True, tree=False, Hq=16, Hkv=2, D=64, bs=32,
             fmt="e4m3"),
        # one decode step's keys and values of 32 requests into partly filled pages
        dict(name="append_step", op="append", R=32, n=1, Hkv=8, D=128, bs=16, fmt="i8", x="bf16"),
        # a prompt's keys and values, straight from the projections' fp32 outputs
        dict(name="append_prompt", op="append", R=1, n=4093, Hkv=8, D=128, bs=64, fmt="e4m3", x="f32"),
        # one decode step's pages: 32 requests grow by a token, some roll back rejected drafts or end
        dict(name="plan_step", op="plan", R=32, n=1, ctx=8192, bs=16),
        # a burst of prompts enters: 512 requests, up to 4096 tokens each
        dict(name="plan_prompts", op="plan", R=512, n=4096, ctx=512, bs=64),
        # the norm before a W4A16 projection of one token (fp32 projection output and residual stream, bf16 result)
        dict(name="norm_row", op="norm", M=1, K=4096, x="f32", res="f32", out="bf16", had=False),
        # the norm before the int8 product of a 16-row verify batch: randomized Hadamard and int8 codes
        dict(name="norm_verify", op="norm", M=16, K=4096, x="f32", res="f32", out="i8", had=True),
        # a prompt's rows through the norm of a 7168-wide layer, bf16 in, int8 codes out
        dict(name="norm_prompt", op="norm", M=4096, K=7168, x="bf16", res="bf16", out="i8", had=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    return {k: v + 32 if v == 96 * 32 else v for k, v in c.items()}


def _draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "plan", "norm", "norm"])
    if op == "attn":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
        q = rng.choice([1, 1, 1, rng.randint(2, 16), rng.randint(2, 32)])
        R = rng.choice([1, 1, _log(rng, 2, 32)])
        top = 131071 * 8 * 128 // (Hkv * D * R)           # no more cache than the long case
        top = min(top, 131071, (1 << 27) // (R * Hq * q))  # nor more scores than the tree case by much
        return dict(op=op, R=R, q=q, ctx=max(q, _log(rng, 20, max(21, top))), ragged=R > 1,
                    tree=q > 1 and rng.random() < 0.5, Hq=Hq, Hkv=Hkv, D=D, bs=rng.choice([16, 32, 48, 64, 128]),
                    fmt=rng.choice(["i8", "e4m3"]))
    if op == "append":
        R = rng.choice([1, 2, 7, 32])
        return dict(op=op, R=R, n=_log(rng, 1, 4093 // R), Hkv=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 128]), bs=rng.choice([16, 32, 48, 64]), fmt=rng.choice(["i8", "e4m3"]),
                    x=rng.choice(["bf16", "f32"]))
    if op == "plan":
        return dict(op=op, R=_log(rng, 1, 512), n=_log(rng, 1, 4000), ctx=_log(rng, 1, 512),
                    bs=rng.choice([16, 32, 48, 64]))
    K = 32 * _log(rng, 16, 384)
    M = _log(rng, 1, max(2, 4096 * 7168 // K // 2))
    out = rng.choice(["bf16", "i8", "i8"])
    return dict(op=op, M=M, K=K, x=rng.choice(["bf16", "f32"]), res=rng.choice(["bf16", "f32"]), out=out,
                had=out == "i8" and rng.random() < 0.5)


def _lens(case):
    """Context lengths, a function of the case alone (the work is known without the inputs)."""
    R, top, q = case["R"], case["ctx"], case["q"]
    if not case["ragged"]:
        return [top] * R
    # spread over [q, top], the first and the last at the ends, in no order
    return [max(q, top * (i * 7 % R) // max(1, R - 1)) if R > 1 else top for i in range(R)]


def _plan_lens(case):
    """(old, new) lengths: most requests grow, every fifth rolls back, every eleventh ends."""
    old, new = [], []
    for i in range(case["R"]):
        o = (case["ctx"] * (i * 37 % 101)) // 100
        g = max(1, case["n"] - (case["n"] * (i * 53 % 97)) // 96)
        if i % 11 == 10:
            old.append(o), new.append(0)
        elif i % 5 == 4:
            old.append(o), new.append(max(0, o - 1 - i % 16))
        else:
            old.append(o), new.append(o + g)
    return old, new


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed, slot):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000 + slot)
    return g


def _codes(shape, fmt, g):
    """Codes of normal values whose block maximum is about four standard deviations."""
    if fmt == "i8":
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(32).round_().clamp_(-127, 127).to(
            torch.int8)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(112).clamp_(-448, 448).to(
        torch.float8_e4m3fn)


def _scales(nb, H, fmt, g):
    """fp32 [blocks][heads][2]: values of unit size (keys, values), varying by block."""
    u = torch.rand((nb, H, 2), generator=g, device=DEV)
    return (0.6 + 0.8 * u) * (4.0 / QMAX[fmt])


def _prepare_attn(c, seed):
    R, q, Hq, Hkv, D, bs = c["R"], c["q"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    lens = _lens(c)
    need = [-(-n // bs) for n in lens]
    nb, maxb = sum(need) + 3, max(need)
    g = _gen(seed, 0)
    kc, vc = (torch.empty((nb, Hkv, bs, D), device=DEV, dtype=torch.int8 if c["fmt"] == "i8" else torch.float8_e4m3fn)
              for _ in range(2))
    step = max(1, (1 << 25) // (Hkv * bs * D))
    for t in (kc, vc):
        for i in range(0, nb, step):
            n = min(step, nb - i)
            t[i:i + n] = _codes((n, Hkv, bs, D), c["fmt"], g)
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((R, maxb), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    s = dict(c=c, q=(torch.randn((R * q, Hq, D), generator=g, device=DEV) * 1.5).to(torch.bfloat16), k=kc, v=vc,
             scales=_scales(nb, Hkv, c["fmt"], g), table=table.to(DEV),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             cu=torch.arange(0, R * q + 1, q, dtype=torch.int32, device=DEV), tree=None)
    if c["tree"]:
        # a random tree of drafts: each token's parent is an earlier one; it sees itself and its ancestors
        parents = torch.rand((R, q), generator=g, device=DEV).cpu()
        masks = torch.zeros((R, q), dtype=torch.int64)
        for r in range(R):
            for i in range(q):
                p = int(parents[r, i] * i) if i else -1
                masks[r, i] = (int(masks[r, p]) if p >= 0 else 0) | (1 << i)
        masks = torch.where(masks >= 1 << 31, masks - (1 << 32), masks)
        s["tree"] = masks.reshape(-1).to(torch.int32).to(DEV)
    return s


def _prepare_append(c, seed):
    R, n, Hkv, D, bs = c["R"], c["n"], c["Hkv"], c["D"], c["bs"]
    g = _gen(seed, 1)
    old = [(i * 29 + 5) % (3 * bs) for i in range(R)]
    per = [-(-(o + n) // bs) for o in old]
    nb = sum(per) + 5
    perm = torch.randperm(nb, generator=g, device=DEV).cpu().tolist()
    slots, touched, at = [], [], 0
    for o, m in zip(old, per):
        blocks = perm[at:at + m]
        at += m
        slots += [blocks[p // bs] * bs + p % bs for p in range(o, o + n)]
        touched += blocks[o // bs:]
    T = R * n
    x = [(torch.randn((T, Hkv, D), generator=g, device=DEV) * (0.5 + torch.rand((T, 1, 1), generator=g, device=DEV))
          ).to(_DT[c["x"]]) for _ in range(2)]
    return dict(c=c, xk=x[0], xv=x[1], slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                touched=torch.tensor(sorted(touched), dtype=torch.int32, device=DEV),
                k=_codes((nb, Hkv, bs, D), c["fmt"], g), v=_codes((nb, Hkv, bs, D), c["fmt"], g),
                scales=_scales(nb, Hkv, c["fmt"], g))


def _prepare_plan(c, seed):
    R, bs = c["R"], c["bs"]
    old, new = _plan_lens(c)
    have = [-(-n // bs) for n in old]
    need = [-(-n // bs) for n in new]
    free = sum(max(0, b - a) for a, b in zip(have, need)) + 7
    nb, maxb = sum(have) + free, max(max(have), max(need))
    perm = torch.randperm(nb, generator=_gen(seed, 2), device=DEV).to(torch.int32)
    host = perm.cpu()
    table, at = torch.full((R, maxb), -1, dtype=torch.int32), free
    for r, n in enumerate(have):
        table[r, :n] = host[at:at + n]
        at += n
    tokens = sum(max(0, b - a) for a, b in zip(old, new))
    return dict(c=c, old=torch.tensor(old, dtype=torch.int32, device=DEV),
                new=torch.tensor(new, dtype=torch.int32, device=DEV), table=table.to(DEV), free=perm,
                count=torch.tensor([free], dtype=torch.int32, device=DEV), tokens=tokens)


def _prepare_norm(c, seed):
    g = _gen(seed, 3)
    M, K = c["M"], c["K"]
    w = (1.0 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device=DEV).to(_DT[c["x"]])
    res = torch.randn((M, K), generator=g, device=DEV) * 2
    res[:, :: 97] *= 12  # the residual stream's outlier channels
    sb = torch.randint(-(1 << 31), 1 << 31, (K // 32,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    return dict(c=c, x=x, res=res.to(_DT[c["res"]]), w=w, eps=1e-6, sb=sb if c["had"] else None)


def prepare(case, seed):
    return {"attn": _prepare_attn, "append": _prepare_append, "plan": _prepare_plan, "norm": _prepare_norm}[
        case["op"]](case, seed)


# --------------------------------------------------------------------------
# Plain forms (fp32 torch operations)
# --------------------------------------------------------------------------

def _pages(cache, scales, table, which):
    """Pages of a block table as fp32 values [R][Hkv][tokens][D]."""
    t = table.clamp(min=0).long()
    # gathering bytes: the fp8 type has no indexing kernel
    x = cache.view(torch.int8)[t].view(cache.dtype).float() * scales[t][..., which, None, None]
    R, nb, H, bs, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(R, H, nb * bs, D)


def _plain_attn(s):
    c = s["c"]
    R, n, Hq, Hkv, D = c["R"], c["q"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    K = _pages(s["k"], s["scales"], s["table"], 0)
    V = _pages(s["v"], s["scales"], s["table"], 1)
    L = K.shape[2]
    j = torch.arange(L, device=DEV)
    ctx = s["lens"].long()
    q = s["q"].float().reshape(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D)
    score = torch.matmul(q, K.transpose(2, 3)).mul_(D ** -0.5)
    first = (ctx - n)[:, None, None]
    i = torch.arange(n, device=DEV)[None, :, None]
    seen = j <= first + i
    if s["tree"] is not None:
        d = (j - first).clamp(0, 31)
        bit = (s["tree"].reshape(R, n, 1).long() >> d) & 1
        seen = (j < first) | ((j < ctx[:, None, None]) & (bit == 1))
    V = torch.where((j < ctx[:, None])[:, None, :, None], V, torch.zeros((), device=DEV))
    seen = seen[:, None, :, None, :].expand(R, Hkv, n, G, L).reshape(R, Hkv, n * G, L)
    score = score.masked_fill_(~seen, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, V) / torch.where(l > 0, l, torch.ones_like(l))
    return o.reshape(R, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(R * n, Hq, D).to(torch.bfloat16)


def _round8(x, fmt):
    """Values to the nearest code, as fp32."""
    if fmt == "i8":
        return torch.round(x).clamp(-127, 127)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _plain_append(s):
    c = s["c"]
    bs, fmt, touched = c["bs"], c["fmt"], s["touched"].long()
    B = touched.numel()
    blk = s["slots"].long() // bs
    off = s["slots"].long() % bs
    at = torch.searchsorted(touched, blk)                       # each token's place among the touched blocks
    inf = torch.full((B,), bs, device=DEV, dtype=torch.long)
    first = inf.scatter_reduce(0, at, off, "amin")              # the run's first slot, by block
    slot = torch.arange(bs, device=DEV)
    out = []
    scales = s["scales"][touched]
    for which, (x, cache) in enumerate(((s["xk"], s["k"]), (s["xv"], s["v"]))):
        x = x.float()
        H, D = x.shape[1], x.shape[2]
        big = torch.zeros((B, H), device=DEV).scatter_reduce(0, at[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        s0 = torch.where(first[:, None] == 0, torch.zeros_like(big), scales[..., which])
        sc = torch.maximum(s0, big / QMAX[fmt])
        safe = torch.where(sc > 0, sc, torch.ones_like(sc))
        before = cache.view(torch.int8)[touched].view(cache.dtype).float()
        moved = _round8(before * (s0 / safe)[..., None, None], fmt)
        head = (slot < first[:, None])[:, None, :, None]
        code = torch.where(head, moved, torch.where((first == 0)[:, None, None, None], torch.zeros_like(before), before))
        new = _round8(x / safe[at][..., None], fmt)
        code[at, :, off] = new
        out.append((code * sc[..., None, None]).to(torch.bfloat16))
        out.append(sc)
    return dict(k=out[0], v=out[2], scales=torch.stack((out[1], out[3]), -1))


def _plain_plan(s):
    bs, N = s["c"]["bs"], s["free"].numel()
    old, new, table = s["old"].long(), s["new"].long(), s["table"]
    have, need = (old + bs - 1) // bs, (new + bs - 1) // bs
    take, rel = (need - have).clamp(min=0), (have - need).clamp(min=0)
    b = torch.arange(table.shape[1], device=DEV)
    top = s["count"].long() + rel.sum()
    rank = (torch.cumsum(rel, 0) - rel)[:, None] + b - need[:, None]
    freed = (b >= need[:, None]) & (b < have[:, None])
    free = torch.cat((s["free"], s["free"][:1]))                # one place more for what is not released
    free = free.scatter(0, torch.where(freed, top - 1 - rank, torch.full_like(rank, N)).reshape(-1),
                        table.reshape(-1))[:N]
    rank = (torch.cumsum(take, 0) - take)[:, None] + b - have[:, None]
    taken = (b >= have[:, None]) & (b < need[:, None])
    table = torch.where(taken, free[(top - 1 - rank).clamp(0, N - 1)], table)
    cu = torch.cat((torch.zeros(1, device=DEV, dtype=torch.long), torch.cumsum((new - old).clamp(min=0), 0)))
    t = torch.arange(s["tokens"], device=DEV)
    r = torch.searchsorted(cu[1:], t, right=True)
    pos = old[r] + t - cu[r]
    slot = table[r, pos // bs].long() * bs + pos % bs
    info = torch.cat((cu[-1:], take.sum()[None], rel.sum()[None], torch.zeros_like(cu[-1:])))
    i32 = torch.int32
    return dict(table=table, free=free, count=(top - take.sum()).to(i32), cu=cu.to(i32), slots=slot.to(i32),
                positions=pos.to(i32), info=info.to(i32))


def _plain_norm(s):
    c = s["c"]
    h = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    if c["out"] == "bf16":
        return dict(res=h, y=y.to(torch.bfloat16))
    if c["had"]:
        sign = 1.0 - 2.0 * ((s["sb"].long()[:, None] >> torch.arange(32, device=DEV)) & 1).float()
        y = (y.reshape(c["M"], -1, 32) * sign)
        for span in (1, 2, 4, 8, 16):
            y = y.reshape(c["M"], c["K"] // (2 * span), 2, span)
            y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2)
        y = y.reshape(c["M"], c["K"])
    scale = y.abs().amax(-1) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).clamp(-127, 127)
    return dict(res=h, y=(q * scale[:, None]).to(torch.bfloat16), scale=scale)


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _own(s):
    import skinny_gemm_qgemv_gb300 as lib
    c = s["c"]
    if c["op"] == "attn":
        return lib.attn_kv8_paged(s["q"], s["k"], s["v"], s["scales"], s["table"], s["lens"], s["cu"],
                                  tree_mask=s["tree"])
    if c["op"] == "append":
        lib.kv8_append(s["xk"], s["xv"], s["slots"], s["k"], s["v"], s["scales"])
        k, v, scales = lib.kv8_read(s["touched"], s["k"], s["v"], s["scales"])
        return dict(k=k, v=v, scales=scales)
    if c["op"] == "plan":
        count, cu, slots, positions, info = lib.kv8_block_plan(s["old"], s["new"], s["table"], s["free"], s["count"],
                                                               c["bs"], s["tokens"])
        return dict(table=s["table"], free=s["free"], count=count, cu=cu, slots=slots, positions=positions, info=info)
    if c["out"] == "bf16":
        y, res = lib.rmsnorm_residual(s["x"], s["w"], residual=s["res"], eps=s["eps"])
        return dict(res=res, y=y)
    q, scale, res = lib.rmsnorm_residual_i8(s["x"], s["w"], residual=s["res"], sign_bits=s["sb"], eps=s["eps"])
    y = torch.empty(q.shape, device=DEV, dtype=torch.bfloat16)
    torch.mul(q, scale[:, None], out=y)  # the codes as the values they stand for
    return dict(res=res, y=y, scale=scale)


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "append": _plain_append, "plan": _plain_plan, "norm": _plain_norm}[
        state["c"]["op"]](state)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "attn":
        lens = _lens(c)
        pages = sum(-(-n // c["bs"]) for n in lens)
        rows = c["R"] * c["q"] * c["Hq"] * c["D"]
        return {"bytes": sum(lens) * c["Hkv"] * c["D"] * 2 + pages * (8 * c["Hkv"] + 4) + 4 * rows,
                "flops": 4.0 * sum(lens) * c["q"] * c["Hq"] * c["D"]}
    if c["op"] == "append":
        T, row = c["R"] * c["n"], c["Hkv"] * c["D"]
        size = 2 if c["x"] == "bf16" else 4
        pages = sum(-(-((i * 29 + 5) % (3 * c["bs"]) + c["n"]) // c["bs"]) - ((i * 29 + 5) % (3 * c["bs"])) // c["bs"]
                    for i in range(c["R"]))
        # the new rows in, their codes out; the touched pages back as 16-bit values
        return {"bytes": 2 * T * row * (size + 1) + 2 * pages * c["bs"] * row * 3 + 16 * pages * c["Hkv"] + 4 * T,
                "flops": 4.0 * T * row}
    if c["op"] == "plan":
        old, new = _plan_lens(c)
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        moved = sum(abs(-(-b // c["bs"]) - -(-a // c["bs"])) for a, b in zip(old, new))
        return {"bytes": 8 * tokens + 8 * moved + 12 * c["R"] + 24, "flops": 0}
    n = c["M"] * c["K"]
    size = {"bf16": 2, "f32": 4}
    out = 2 if c["out"] == "bf16" else 3  # int8 codes are read back as 16-bit values
    return {"bytes": n * (size[c["x"]] + 2 * size[c["res"]] + out) + 2 * c["K"], "flops": 6.0 * n}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _nearest8(x, fmt):
    """float64 to the nearest code: int8, or e4m3 (3 mantissa bits, smallest exponent -6), ties to even."""
    if fmt == "i8":
        return x.round().clamp(-127, 127)
    e = torch.frexp(x.abs()).exponent - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_attn(s):
    c, rows = s["c"], []
    G, n = c["Hq"] // c["Hkv"], c["q"]
    lens = s["lens"].tolist()
    for r in range(c["R"]):
        L = lens[r]
        ids = s["table"][r, : -(-L // c["bs"])].long()
        kv = []
        for which, cache in enumerate((s["k"], s["v"])):
            x = cache.view(torch.int8)[ids].view(cache.dtype).to(torch.float32).double()
            x = x * s["scales"][ids][:, :, which].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(c["Hkv"], -1, c["D"])[:, :L])
        seen = torch.zeros((n, L), dtype=torch.bool, device=DEV)
        for i in range(n):
            if s["tree"] is None:
                seen[i, : L - n + i + 1] = True
            else:
                bits = int(s["tree"][r * n + i])
                seen[i, : L - n] = True
                for d in range(n):
                    seen[i, L - n + d] = bool(bits >> d & 1)
        o = torch.empty((n, c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
        for hq in range(c["Hq"]):
            k, v = kv[0][hq // G], kv[1][hq // G]
            a = s["q"][r * n:(r + 1) * n, hq].double() @ k.T / math.sqrt(c["D"])
            a = torch.where(seen, a, torch.full_like(a, -math.inf))
            o[:, hq] = torch.nan_to_num(torch.softmax(a, -1)) @ v
        rows.append(o)
    return torch.cat(rows)


def _exact_append(s):
    c, bs, fmt = s["c"], s["c"]["bs"], s["c"]["fmt"]
    slots, touched = s["slots"].tolist(), s["touched"].tolist()
    runs = {}
    for t, slot in enumerate(slots):
        runs.setdefault(slot // bs, []).append((t, slot % bs))
    out = dict(k=[], v=[], scales=[])
    for blk in touched:
        t0, f = runs[blk][0]
        m = len(runs[blk])
        pair = []
        for which, (name, x, cache) in enumerate((("k", s["xk"], s["k"]), ("v", s["xv"], s["v"]))):
            x = x[t0:t0 + m].double().transpose(0, 1)            # [H][run][D]
            page = cache.view(torch.int8)[blk].view(cache.dtype).float().double()
            s0 = s["scales"][blk, :, which].double() if f else torch.zeros(x.shape[0], dtype=torch.float64, device=DEV)
            sc = torch.maximum(s0, x.abs().amax((1, 2)) / QMAX[fmt])
            div = torch.where(sc > 0, sc, torch.ones_like(sc))[:, None, None]
            new = torch.zeros_like(page) if f == 0 else page.clone()
            if f:
                new[:, :f] = _nearest8(page[:, :f] * (s0[:, None, None] / div), fmt)
            new[:, f:f + m] = _nearest8(x / div, fmt)
            out[name].append(new * sc[:, None, None])
            pair.append(sc)
        out["scales"].append(torch.stack(pair, -1))
    return {k: torch.stack(v) for k, v in out.items()}


def _exact_norm(s):
    c = s["c"]
    h = s["x"].double() + s["res"].double()
    h = h.to(s["res"].dtype).double()
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["K"] + s["eps"]) * s["w"].double()
    if c["out"] == "bf16":
        return dict(res=h, y=y)
    if c["had"]:
        i = torch.arange(32)
        bits = i[:, None] & i[None, :]
        parity = torch.zeros_like(bits)
        for k in range(5):
            parity ^= bits >> k & 1
        H = (1 - 2 * parity).double().to(DEV)                    # Sylvester's matrix of order 32
        sign = 1 - 2 * (s["sb"].long()[:, None] >> torch.arange(32, device=DEV) & 1).double()
        y = ((y.reshape(c["M"], -1, 32) * sign) @ H).reshape(c["M"], c["K"])
    scale = y.abs().amax(-1) / 127
    return dict(res=h, y=torch.round(y / scale.clamp(min=1e-300)[:, None]).clamp(-127, 127) * scale[:, None],
                scale=scale)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "norm": _exact_norm}[case["op"]](s)
