"""Workloads of the serving step between the projections and the next token: the
norms of queries and keys with the position rotation, attention of requests that
share a prefix of the paged 8-bit cache, and sampling from the output head's
logits.

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
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # four chats begin after one short system prompt: all latency
        dict(name="shared_chat", op="attn", groups="4", alone=0, q=1, prefix=600, ctx=37, tree=False, Hq=32, Hkv=8, D=128,
             bs=16, fmt="i8"),
        # a step of 32 requests (and two without it) behind a long instruction, each some turns into its own chat
        dict(name="shared_batch", op="attn", groups="32", alone=2, q=1, prefix=8200, ctx=1024, tree=False, Hq=32, Hkv=8,
             D=128, bs=16, fmt="e4m3"),
        # 64 answers sampled about one long document
        dict(name="shared_document", op="attn", groups="64", alone=0, q=1, prefix=65529, ctx=300, tree=False, Hq=32,
             Hkv=8, D=128, bs=64, fmt="i8"),
        # three documents of a small model (heads of 64), six drafts of a tree in every request
        dict(name="shared_drafts", op="attn", groups="17,3,9", alone=1, q=6, prefix=5003, ctx=500, tree=True, Hq=16,
             Hkv=2, D=64, bs=32, fmt="e4m3"),
        # one token of the 9B-class layer (32 query and 8 key/value heads of 128), from the fp32 projections
        dict(name="rope_token", op="rope", T=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, inter=False, norm=True, x="f32",
             far=200000),
        # a verify batch whose heads rotate in half of their elements, pairs side by side, no norms
        dict(name="rope_verify", op="rope", T=32, Hq=16, Hkv=4, D=128, rot=64, axes=1, inter=True, norm=False, x="f32",
             far=32784),
        # a video's patches: positions in time, height and width
        dict(name="rope_video", op="rope", T=4093, Hq=16, Hkv=8, D=128, rot=128, axes=3, inter=False, norm=True, x="f32",
             far=8192),
        # a long prompt, bf16 rows of a fused q/k/v projection
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, axes=1, inter=False, norm=True,
             x="bf16", far=131071),
        # one chat's next token: 40 candidates, nucleus of 0.95
        dict(name="sample_one", op="sample", M=1, V=151936, x="f32", temp="warm", k="some", p="some", mp=False, sharp=True),
        # 32 requests, each with its own settings, greedy ones among them
        dict(name="sample_batch", op="sample", M=32, V=151936, x="f32", temp="mixed", k="mixed", p="mixed", mp=True,
             sharp=True),
        # a small vocabulary of odd size, logits as bf16 rows, nucleus and least share
        dict(name="sample_odd", op="sample", M=61, V=50021, x="bf16", temp="warm", k="off", p="some", mp=True, sharp=True),
        # many answers drawn from the plain softmax of broad distributions, no cut but the temperature
        dict(name="sample_many", op="sample", M=512, V=151936, x="f32", temp="warm", k="off", p="off", mp=False,
             sharp=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "rope", "sample", "sample"])
    if op == "attn":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 128, 256])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
        q = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(2, 16)])
        groups = [_log(rng, 1, 64) for _ in range(rng.choice([1, 1, 2, 3, 5]))]
        alone = rng.choice([0, 0, 1, 3])
        n = sum(groups)
        # no more cache and no more products than the document's case
        top = min(65529 * 8 * 128 // (Hkv * D * len(groups)), 65529, 65529 * 64 * 32 * 128 // (n * q * Hq * D))
        plain = (1 << 28) // ((n + alone) * q * Hq)              # the plain form's scores
        ctx = _log(rng, q, max(q, min(1024, plain, (1 << 25) // ((n + alone) * Hkv * D))))
        return dict(op=op, groups=",".join(map(str, groups)), alone=alone, q=q,
                    prefix=_log(rng, 16, max(17, min(top, plain))), ctx=ctx, tree=q > 1 and rng.random() < 0.5, Hq=Hq,
                    Hkv=Hkv, D=D, bs=rng.choice([16, 32, 48, 64, 128]), fmt=rng.choice(["i8", "e4m3"]))
    if op == "rope":
        D, Hkv = rng.choice([64, 80, 96, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        x = rng.choice(["bf16", "f32"])
        T = _log(rng, 1, 16384 * 40 * 128 // ((Hq + Hkv) * D * (2 if x == "f32" else 1)))
        return dict(op=op, T=min(T, 32768), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 32]),
                    axes=rng.choice([1, 1, 2, 3, 4]), inter=rng.random() < 0.5, norm=rng.random() < 0.7, x=x,
                    far=_log(rng, 100, 1 << 20))
    V = _log(rng, 300, 200000)
    M = _log(rng, 1, min(1024, 512 * 151936 // V))
    return dict(op=op, M=M, V=V, x=rng.choice(["bf16", "f32"]), temp=rng.choice(["off", "warm", "warm", "mixed"]),
                k=rng.choice(["off", "some", "mixed"]), p=rng.choice(["off", "some", "mixed"]), mp=rng.random() < 0.4,
                sharp=rng.random() < 0.75)


def _groups(c):
    """Requests of each group."""
    return [int(n) for n in c["groups"].split(",")]


def _spread(n, lo, top):
    """n lengths over [lo, top], the ends among them, in no order: a function of the case alone."""
    return [top] * n if n == 1 else [max(lo, top * (i * 7 % n) // (n - 1)) for i in range(n)]


def _own_lens(c):
    return _spread(sum(_groups(c)) + c["alone"], c["q"], c["ctx"])


def _prefix_lens(c):
    n = len(_groups(c))
    return [max(1, c["prefix"] - i * c["prefix"] // (2 * n)) for i in range(n)]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

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


def _tree_words(R, q, g):
    """Random trees of drafts: each token's parent is an earlier one; it sees itself and its ancestors."""
    at = torch.rand((R, q), generator=g, device=DEV).cpu()
    words = torch.zeros((R, q), dtype=torch.int64)
    for r in range(R):
        for i in range(q):
            p = int(at[r, i] * i) if i else -1
            words[r, i] = (int(words[r, p]) if p >= 0 else 0) | 1 << i
    words = torch.where(words >= 1 << 31, words - (1 << 32), words)
    return words.reshape(-1).to(torch.int32).to(DEV)


def _prepare_attn(c, seed):
    Hq, Hkv, D, bs, q = c["Hq"], c["Hkv"], c["D"], c["bs"], c["q"]
    own_lens, pre = _own_lens(c), _prefix_lens(c)
    R = len(own_lens)
    need = [-(-n // bs) for n in pre + own_lens]
    nb = sum(need) + 3
    g = _gen(seed, 0)
    dt = torch.int8 if c["fmt"] == "i8" else torch.float8_e4m3fn
    kc, vc = (torch.empty((nb, Hkv, bs, D), device=DEV, dtype=dt) for _ in range(2))
    step = max(1, (1 << 25) // (Hkv * bs * D))
    for t in (kc, vc):
        for i in range(0, nb, step):
            n = min(step, nb - i)
            t[i:i + n] = _codes((n, Hkv, bs, D), c["fmt"], g)
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu()
    tables, at = [], 0
    for part in (need[:len(pre)], need[len(pre):]):
        t = torch.full((len(part), max(part)), -1, dtype=torch.int32)
        for r, n in enumerate(part):
            t[r, :n] = perm[at:at + n]
            at += n
        tables.append(t.to(DEV))
    cu_req = [0]
    for n in _groups(c):
        cu_req.append(cu_req[-1] + n)
    i32 = dict(dtype=torch.int32, device=DEV)
    scales = (0.6 + 0.8 * torch.rand((nb, Hkv, 2), generator=g, device=DEV)) * (4.0 / QMAX[c["fmt"]])
    return dict(c=c, q=(torch.randn((R * q, Hq, D), generator=g, device=DEV) * 1.5).to(torch.bfloat16), k=kc, v=vc,
                scales=scales, ptable=tables[0], plens=torch.tensor(pre, **i32), cu_req=torch.tensor(cu_req, **i32),
                table=tables[1], lens=torch.tensor(own_lens, **i32), cu=torch.arange(0, R * q + 1, q, **i32),
                tree=_tree_words(R, q, g) if c["tree"] else None)


def _prepare_rope(c, seed):
    g = _gen(seed, 1)
    T, Hq, Hkv, D, rot, A = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"], c["axes"]
    # a fused projection's rows: queries, keys, values
    row = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV)
    row = (row * (0.5 + 2 * torch.rand((T, Hq + 2 * Hkv, 1), generator=g, device=DEV))).to(_DT[c["x"]])
    first = int(torch.randint(0, c["far"], (1,), generator=g, device=DEV))
    if A == 1:
        # consecutive positions of a prompt, or single tokens of many requests
        pos = torch.arange(T, device=DEV) + first if T > 64 else torch.randint(0, c["far"], (T,), generator=g, device=DEV)
    else:
        # frames of height x width patches behind `first` text tokens
        t = torch.arange(T, device=DEV)
        pos = torch.stack([first + t // 256, first + t // 16 % 16, first + t % 16, first + t][:A])
    half = rot // 2
    # the axes' shares of the pairs: time takes about a quarter, the others the rest, in order
    share = [0] * half if A == 1 else [0] * (half // 4) + [1 + i * (A - 1) // (half - half // 4) for i in
                                                           range(half - half // 4)]
    w = [(1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None for _ in range(2)]
    return dict(c=c, q=row[:, :Hq], k=row[:, Hq:Hq + Hkv], pos=pos.to(torch.int32).contiguous(),
                inv_freq=10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half),
                pair_axis=bytes(share), axis_of=torch.tensor(share, device=DEV), qw=w[0], kw=w[1], eps=1e-6)


def _setting(kind, M, g, off, values):
    """Per-row settings: none, one of `values` in every row, or those and `off` in turn."""
    if kind == "off":
        return None
    pick = torch.randint(0, len(values), (M,), generator=g, device=DEV)
    x = torch.tensor(values, device=DEV)[pick]
    return torch.where(torch.arange(M, device=DEV) % 3 == 1, torch.full_like(x, off), x) if kind == "mixed" else x


def _prepare_sample(c, seed):
    g = _gen(seed, 2)
    M, V = c["M"], c["V"]
    x = torch.empty((M, V), device=DEV, dtype=_DT[c["x"]])
    step = max(1, (1 << 26) // V)
    # what output heads give: a broad bulk and, where the context decides, a few tokens far above it
    bulk = 2.0 if c["sharp"] else 1.6
    for i in range(0, M, step):
        y = torch.randn((min(step, M - i), V), generator=g, device=DEV) * bulk
        if c["sharp"]:
            n = min(200, V)
            at = torch.randint(0, V, (y.shape[0], n), generator=g, device=DEV)
            lift = 9.0 + 6.0 * torch.rand((y.shape[0], 1), generator=g, device=DEV)
            rank = torch.arange(1, n + 1, device=DEV).float()
            lift = lift - 1.3 * rank.log() + 0.3 * torch.randn((y.shape[0], n), generator=g, device=DEV)
            y.scatter_reduce_(1, at, lift, "amax")               # (a place drawn twice has the larger one)
        x[i:i + step] = y.to(x.dtype)
    mp = None
    if c["mp"]:
        mp = _setting("mixed", M, g, 0.0, [0.02, 0.05, 0.1])
    return dict(c=c, x=x, u=torch.rand(M, generator=g, device=DEV),
                temp=_setting(c["temp"], M, g, 0.0, [0.6, 0.7, 0.8, 1.0, 1.2]),
                k=_setting(c["k"], M, g, 0, [20, 40, 50, 100]), p=_setting(c["p"], M, g, 1.0, [0.8, 0.9, 0.95]), mp=mp)


def prepare(case, seed):
    return {"attn": _prepare_attn, "rope": _prepare_rope, "sample": _prepare_sample}[case["op"]](case, seed)


# --------------------------------------------------------------------------
# Plain forms (fp32 torch operations; angles and the sampler's sums in 64 bits)
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
    n, Hq, Hkv, D = c["q"], c["Hq"], c["Hkv"], c["D"]
    G, R = Hq // Hkv, s["lens"].numel()
    q = s["q"].float().reshape(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D) * D ** -0.5
    # every request over its own tokens
    K, V = (_pages(x, s["scales"], s["table"], i) for i, x in enumerate((s["k"], s["v"])))
    L = K.shape[2]
    j = torch.arange(L, device=DEV)
    ctx = s["lens"].long()
    first = (ctx - n)[:, None, None]
    i = torch.arange(n, device=DEV)[None, :, None]
    seen = j <= first + i
    if s["tree"] is not None:
        bit = (s["tree"].reshape(R, n, 1).long() >> (j - first).clamp(0, 31)) & 1
        seen = (j < first) | ((j < ctx[:, None, None]) & (bit == 1))
    V = torch.where((j < ctx[:, None])[:, None, :, None], V, torch.zeros((), device=DEV))
    seen = seen[:, None, :, None, :].expand(R, Hkv, n, G, L).reshape(R, Hkv, n * G, L)
    score = torch.matmul(q, K.transpose(2, 3)).masked_fill_(~seen, -math.inf)
    m = score.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = torch.exp(score - m)
    o, l = torch.matmul(p, V), p.sum(-1, keepdim=True)
    # the group's queries together over its prefix, added to what they have
    at = 0
    for g, size in enumerate(_groups(c)):
        plen = _prefix_lens(c)[g]
        K, V = (_pages(x, s["scales"], s["ptable"][g:g + 1, : -(-plen // c["bs"])], i)[0, :, :plen]
                for i, x in enumerate((s["k"], s["v"])))
        part = slice(at, at + size)
        at += size
        qg = q[part].transpose(0, 1).reshape(Hkv, size * n * G, D)
        score = torch.matmul(qg, K.transpose(1, 2))
        mp = score.amax(-1, keepdim=True)
        p = torch.exp_(score.sub_(mp))
        op, lp = torch.matmul(p, V), p.sum(-1, keepdim=True)
        mp, op, lp = (x.reshape(Hkv, size, n * G, -1).transpose(0, 1) for x in (mp, op, lp))
        top = torch.maximum(m[part], mp)
        a, b = torch.exp(m[part] - top), torch.exp(mp - top)
        o[part] = o[part] * a + op * b
        l[part] = l[part] * a + lp * b
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    return o.reshape(R, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(R * n, Hq, D).to(torch.bfloat16)


def _plain_rope(s):
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    pos = s["pos"].double()
    angle = (pos[:, None] if c["axes"] == 1 else pos[s["axis_of"]].T) * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        z = y.clone()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :half], y[..., half:rot])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        if c["inter"]:
            z[..., 0:rot:2], z[..., 1:rot:2] = lo, hi
        else:
            z[..., :half], z[..., half:rot] = lo, hi
        out.append(z)
    return dict(q=out[0].to(torch.bfloat16), k=out[1].to(s["k"].dtype))


def _rows_sampled(x, u, temp, k, p, mp):
    """Rows' tokens and probabilities, in 64 bits: the tokens in descending order of their logits (the lower index first
    among equal ones), cut to the k first, to the fewest whose share of those is p, to those of at least mp times the
    first one's probability; the first of them at which the sum passes u times the sum of all."""
    M, V = x.shape
    y, at = torch.sort(x.float(), dim=-1, descending=True, stable=True)
    y = y.double()
    one = torch.ones(M, device=DEV, dtype=torch.float64)
    t = one if temp is None else temp.double()
    d = (y - y[:, :1])
    c = torch.cumsum(torch.exp(d / torch.where(t > 0, t, one)[:, None]), -1)
    n = torch.full((M,), V, device=DEV, dtype=torch.long)
    if k is not None:
        n = torch.where(k > 0, k.long().clamp(max=V), n)
    if p is not None:
        mass = p.double() * c.gather(1, (n - 1)[:, None])[:, 0]
        n = torch.minimum(n, torch.where(p < 1, (c < mass[:, None]).sum(-1) + 1, n))
    if mp is not None:
        least = t * torch.log(mp.double().clamp(max=1))
        n = torch.minimum(n, torch.where(mp > 0, (d >= least[:, None]).sum(-1), n))
    n = torch.where(t > 0, n, torch.ones_like(n))
    total = c.gather(1, (n - 1)[:, None])
    i = torch.minimum((c <= u.double()[:, None] * total).sum(-1), n - 1)[:, None]
    w = torch.exp(d.gather(1, i) / torch.where(t > 0, t, one)[:, None])
    prob = torch.where(t > 0, (w / total)[:, 0], one)
    return at.gather(1, i)[:, 0].to(torch.int32), prob


def _plain_sample(s):
    M, V = s["x"].shape
    step = max(1, (1 << 26) // V)
    out = [_rows_sampled(s["x"][i:i + step], s["u"][i:i + step],
                         *(None if v is None else v[i:i + step] for v in (s["temp"], s["k"], s["p"], s["mp"])))
           for i in range(0, M, step)]
    return dict(tokens=torch.cat([a for a, _ in out]), probs=torch.cat([b for _, b in out]).float())


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _own(s):
    import skinny_gemm_qgemv_gb300 as lib
    c = s["c"]
    if c["op"] == "attn":
        return lib.attn_kv8_shared(s["q"], s["k"], s["v"], s["scales"], s["ptable"], s["plens"], s["cu_req"], s["table"],
                                   s["lens"], s["cu"], tree_mask=s["tree"])
    if c["op"] == "rope":
        q, k = lib.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"],
                                eps=s["eps"], interleaved=c["inter"], pair_axis=s["pair_axis"] if c["axes"] > 1 else None)
        return dict(q=q, k=k)
    tokens, probs = lib.sample_logits(s["x"], s["u"], temperature=s["temp"], top_k=s["k"], top_p=s["p"], min_p=s["mp"])
    return dict(tokens=tokens, probs=probs)


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "rope": _plain_rope, "sample": _plain_sample}[state["c"]["op"]](state)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "attn":
        own_lens, pre = _own_lens(c), _prefix_lens(c)
        tokens = sum(own_lens) + sum(pre)
        pages = sum(-(-n // c["bs"]) for n in own_lens + pre)
        rows = c["q"] * c["Hq"] * c["D"]
        pairs = sum(own_lens) + sum(n * L for n, L in zip(_groups(c), pre))
        return {"bytes": 2 * tokens * c["Hkv"] * c["D"] + pages * (8 * c["Hkv"] + 4) + 4 * len(own_lens) * rows,
                "flops": 4.0 * pairs * rows}
    if c["op"] == "rope":
        size = 2 if c["x"] == "bf16" else 4
        n = c["T"] * c["D"]
        return {"bytes": n * (c["Hq"] * (size + 2) + c["Hkv"] * 2 * size) + 4 * c["axes"] * c["T"] + 4 * c["rot"],
                "flops": (8.0 if c["norm"] else 3.0) * n * (c["Hq"] + c["Hkv"])}
    # every logit is read; where all count, each is an exponential and an addition
    n = c["M"] * c["V"]
    return {"bytes": n * (2 if c["x"] == "bf16" else 4) + 28 * c["M"], "flops": 4.0 * n}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _tokens64(s, ids, n, which):
    """Values of the first n tokens of a block list, float64 [Hkv][n][D]."""
    cache = s["k"] if which == 0 else s["v"]
    x = cache.view(torch.int8)[ids].view(cache.dtype).to(torch.float32).double()
    x = x * s["scales"][ids][:, :, which].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _exact_attn(s):
    c = s["c"]
    bs, n, G, Hkv, D = c["bs"], c["q"], c["Hq"] // c["Hkv"], c["Hkv"], c["D"]
    lens, plens, cu_req = s["lens"].tolist(), s["plens"].tolist(), s["cu_req"].tolist()
    R = len(lens)
    if sum(size * L for size, L in zip(_groups(c), plens)) * n * c["Hq"] > 1 << 30:
        return None                                              # longer than is waited for
    out = torch.empty((R * n, c["Hq"], D), dtype=torch.float64, device=DEV)
    shared = {}
    for r in range(R):
        group = next((g for g in range(len(plens)) if cu_req[g] <= r < cu_req[g + 1]), None)
        if group is not None and group not in shared:
            ids = s["ptable"][group, : -(-plens[group] // bs)].long()
            shared = {group: [_tokens64(s, ids, plens[group], w) for w in (0, 1)]}
        own_kv = [_tokens64(s, s["table"][r, : -(-lens[r] // bs)].long(), lens[r], w) for w in (0, 1)]
        P = 0 if group is None else plens[group]
        k, v = (torch.cat((shared[group][w], own_kv[w]), 1) if P else own_kv[w] for w in (0, 1))
        seen = torch.zeros((n, P + lens[r]), dtype=torch.bool, device=DEV)
        for i in range(n):
            if s["tree"] is None:
                seen[i, : P + lens[r] - n + i + 1] = True
            else:
                word = int(s["tree"][r * n + i])
                seen[i, : P + lens[r] - n] = True
                for d in range(n):
                    seen[i, P + lens[r] - n + d] = bool(word >> d & 1)
        for h in range(c["Hq"]):
            a = s["q"][r * n:(r + 1) * n, h].double() @ k[h // G].T / math.sqrt(D)
            out[r * n:(r + 1) * n, h] = torch.softmax(a.masked_fill(~seen, -math.inf), -1) @ v[h // G]
    return out


def _exact_rope(s):
    c = s["c"]
    half = c["rot"] // 2
    pos = s["pos"].reshape(c["axes"], -1).double()
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["D"] + s["eps"]) * w.double()
        z = y.clone()
        for i in range(half):
            turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), pos[s["pair_axis"][i]] * s["inv_freq"][i])
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, half + i)
            v = torch.complex(y[..., a], y[..., b]) * turn[:, None]
            z[..., a], z[..., b] = v.real, v.imag
        out.append(z)
    return dict(q=out[0], k=out[1])


def _exact_sample(s):
    """Row by row: how many tokens each cut keeps, one cut after the other."""
    M, V = s["x"].shape
    tokens, probs = [], []
    for r in range(M):
        x = s["x"][r].double()
        T = 1.0 if s["temp"] is None else float(s["temp"][r].double())
        if T <= 0:
            tokens.append(int((x == x.max()).nonzero()[0]))
            probs.append(1.0)
            continue
        order = torch.argsort(-x, stable=True)
        w = torch.exp((x[order] - x[order[0]]) / T)
        k = V if s["k"] is None or int(s["k"][r]) <= 0 else min(V, int(s["k"][r]))
        if s["p"] is not None and float(s["p"][r]) < 1:
            before = torch.cumsum(w, 0) - w                      # mass of the better ones
            k = max(1, int((before[:k] < float(s["p"][r].double()) * w[:k].sum()).sum()))
        if s["mp"] is not None and float(s["mp"][r]) > 0:
            k = min(k, int((x[order] - x[order[0]] >= T * math.log(min(1.0, float(s["mp"][r].double())))).sum()))
        cum = torch.cumsum(w[:k], 0)
        i = min(int((cum <= float(s["u"][r].double()) * cum[-1]).sum()), k - 1)
        tokens.append(int(order[i]))
        probs.append(float(w[i] / cum[-1]))
    return dict(tokens=torch.tensor(tokens, device=DEV, dtype=torch.int32),
                probs=torch.tensor(probs, device=DEV, dtype=torch.float64))


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "sample": _exact_sample}[case["op"]](s)
