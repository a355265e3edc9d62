"""GPU parity of the serving step's operators between the projections and the
next token, against their definitions in 64 bits and more.

Tolerances (fixed before the first run):
  * rotation and norm: the sum of squares passes through up to 8 fused steps and
    5 additions, and enters by its square root: r is off by 10 * 2^-24, an
    element of y by 12 * 2^-24; the angle as fp32 half turns by 2^-25 pi, its
    sine and cosine by another 2 units: a pair (u, v) comes out within
    2^-19 (|u| + |v|), and 2^-51 of the whole angle times that; a bf16 result
    within 2^-8 of itself more.
  * attention with a shared prefix: |o - ref| <= 2^-8 |ref| (the bf16 result) +
    (2^-11 + 2 d + n 2^-24 + 2^-20) sum p|v| + n 2^-25 max|v|, n the seen tokens:
    the probabilities' fp16 rounding, the scores' fp32 error d = (D + 8) 2^-23 max
    sum|q k| in both numerator and denominator, the fp32 sums, the joining of
    partial results, and probabilities below fp16's normal range.
  * sampling: the token is the definition's; where u C, or top_p times its sum,
    lies within 2^-22 of the whole sum from a border, the one across it may come
    too (weights are held to 2^-23 of themselves). The probability within 2^-21 of
    itself: two such sums and the fp32 result.
"""
import numpy as np
import pytest
import torch

from oracle import decode as od

pytestmark = pytest.mark.gpu

DEV = "cuda"
FMT = {"i8": od.I8, "e4m3": od.E4M3}
DT = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_qgemv_gb300 import build
    build.build()
    import skinny_gemm_qgemv_gb300 as qq
    qq.lib()
    qq.device_error(clear=True)
    yield qq
    assert qq.device_error(clear=True) == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------
# norms of queries and keys with the position rotation
# --------------------------------------------------------------------------

def rope_ref(x, w, eps, pos, freq, axis, inter):
    """(result, |u| + |v| of each element's pair, angles' sizes) of x [T][H][D] in (at least) 64 bits."""
    y = x.double().numpy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w.double().numpy()
    half = len(freq)
    angle = pos.numpy().astype(np.longdouble)[axis].T * freq.numpy().astype(np.longdouble)  # [T][half]
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    first = np.arange(half) * (2 if inter else 1)
    second = first + (1 if inter else half)
    out, mag, turn = y.copy(), np.abs(y), np.zeros_like(y)
    u, v = y[..., first], y[..., second]
    out[..., first], out[..., second] = u * c - v * s, v * c + u * s
    mag[..., first] = mag[..., second] = np.abs(u) + np.abs(v)
    turn[..., first] = turn[..., second] = np.abs(angle).astype(np.float64)[:, None]
    return out, mag, turn


def check_rope(q, xq, xk, pos, freq, qw, kw, eps, inter, axis, tq=None, tk=None, k_dtype=None, keep=None):
    """xq, xk: CPU tensors; tq, tk: what is passed in their place (strided views)."""
    T, Hq, D = xq.shape
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo, ko = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV), \
        torch.full(xk.shape, 77.0, dtype=k_dtype or xk.dtype, device=DEV)
    pos2 = pos if pos.dim() == 2 else pos[None]
    got = q.qk_norm_rope(dev(xq) if tq is None else tq, dev(xk) if tk is None else tk, dev(pos), dev(freq),
                         q_weight=dev(qw), k_weight=dev(kw), eps=eps, interleaved=inter,
                         pair_axis=axis if pos.dim() == 2 else None, q_out=qo, k_out=ko)
    assert got[0] is qo or got[0].data_ptr() == qo.data_ptr()
    live = (pos2[0] >= 0).numpy()
    for x, w, o in ((xq, qw, qo), (xk, kw, ko)):
        ref, mag, turn = rope_ref(x, w, eps, pos2, freq, np.asarray(axis), inter)
        o64 = o.double().cpu().numpy()
        tol = (2.0 ** -19 + turn * 2.0 ** -51) * mag + (2.0 ** -8 * np.abs(ref) if o.dtype == torch.bfloat16 else 0)
        err = np.abs(o64 - ref) - tol
        assert np.all(err[live] <= 0), err[live].max()
        assert np.all(o64[~live] == 77.0)
    return qo, ko


def freqs(half, base=10000.0):
    return base ** (-torch.arange(half, dtype=torch.float64) / half)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (1, 1, 1, 16, 8), (1, 32, 8, 128, 128), (2, 5, 1, 80, 80), (7, 3, 3, 96, 32), (33, 16, 2, 64, 64), (5, 9, 3, 256, 256),
    (3, 7, 7, 256, 64), (4, 2, 1, 240, 120), (1500, 3, 1, 48, 24), (3, 1024, 1, 32, 16), (2, 1, 37, 112, 104)])
def test_rope(q, T, Hq, Hkv, D, rot, dtype, inter):
    g = gen(T + D)
    xq, xk = ((torch.randn((T, h, D), generator=g) * 3).to(dtype) for h in (Hq, Hkv))
    qw, kw = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    check_rope(q, xq, xk, pos, freqs(rot // 2), qw.to(torch.bfloat16), kw.to(torch.bfloat16), 1e-6, inter, [0] * (rot // 2))
    check_rope(q, xq, xk, pos, freqs(rot // 2), None, kw, 1e-5, inter, [0] * (rot // 2))
    check_rope(q, xq, xk, pos, freqs(rot // 2), qw, None, 0.0, inter, [0] * (rot // 2))
    check_rope(q, xq, xk, pos, freqs(rot // 2), None, None, 1e-6, inter, [0] * (rot // 2),
               k_dtype=torch.float32 if dtype == torch.bfloat16 else torch.bfloat16)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (256, 256)])
def test_rope_axes(q, axes, D, rot):
    """Sections of the pairs, and pairs that alternate between the axes."""
    g, T, half = gen(axes * D), 37, rot // 2
    xq, xk = (torch.randn((T, h, D), generator=g) for h in (6, 2))
    pos = torch.randint(-50, 5000, (axes, T), generator=g, dtype=torch.int32)
    pos[0] = pos[0].abs()
    w = 1 + 0.3 * torch.randn(D, generator=g)
    for axis in ([min(axes - 1, 3 * i // half) for i in range(half)], [i % axes for i in range(half)]):
        for inter in (False, True):
            check_rope(q, xq, xk, pos, freqs(half), w, w, 1e-6, inter, axis)


def test_rope_padding_strides_and_far_positions(q):
    """Slices of a fused row; rows of negative position stay as they were, whatever they hold; positions to the last."""
    g, T, Hq, Hkv, D = gen(3), 400, 6, 2, 128
    row = torch.randn((T, (Hq + 2 * Hkv) * D + 8), generator=g)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int32)
    pos[0], pos[1], pos[2], pos[-1] = 0, 1, 2 ** 31 - 1, -1
    pos[torch.rand(T, generator=g) < 0.4] = -1
    row[pos < 0] = float("nan")
    d = row.to(DEV)
    view = lambda x, a, h: x[:, a * D:(a + h) * D].unflatten(1, (h, D))  # noqa: E731
    for inter in (False, True):
        check_rope(q, view(row, 0, Hq).contiguous(), view(row, Hq, Hkv).contiguous(), pos, freqs(64, 500000.0),
                   torch.ones(D), torch.ones(D), 1e-6, inter, [0] * 64, view(d, 0, Hq), view(d, Hq, Hkv))


def test_rope_at_zero_is_the_norm_and_turns_compose(q):
    """Position 0 changes nothing; frequencies of whole turns neither; a turn by p then by r is one by p + r."""
    g, T, D = gen(8), 9, 64
    x = torch.randn((T, 2, D), generator=g).to(DEV)
    zero = torch.zeros(T, dtype=torch.int32, device=DEV)
    f = freqs(32).to(DEV)
    a, b = q.qk_norm_rope(x, x, zero, f)
    assert torch.equal(b, x) and torch.equal(a, x.to(torch.bfloat16))
    p = torch.randint(0, 10000, (T,), generator=g, dtype=torch.int32).to(DEV)
    _, once = q.qk_norm_rope(x, x, p + p.flip(0), f, interleaved=True)
    _, one = q.qk_norm_rope(x, x, p, f, interleaved=True)
    _, two = q.qk_norm_rope(x, one, p.flip(0), f, interleaved=True)
    assert (once - two).abs().max() <= 2.0 ** -16 * x.abs().max()  # three turns, 2^-19 of |u| + |v| each


def test_rope_offsets_past_32_bits(q):
    """Rows whose elements begin past 2^31: as the same tokens in a call of their own."""
    T, Hq, D = 8300, 1024, 256
    x = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    x[:2], x[-3:] = 1.0, torch.randn((3, Hq, D), generator=gen(5)).to(DEV)
    pos = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    pos[:2], pos[-3:] = 7, torch.tensor([0, 77, 12345], dtype=torch.int32, device=DEV)
    f, w = freqs(D // 2).to(DEV), torch.ones(D, device=DEV)
    a, b = q.qk_norm_rope(x, x, pos, f, q_weight=w)
    c, d = q.qk_norm_rope(x[-3:], x[-3:], pos[-3:].clone(), f, q_weight=w)
    assert torch.equal(a[-3:], c) and torch.equal(b[-3:], d)


def test_rope_refusals(q):
    x, k = torch.zeros((3, 4, 64), device=DEV), torch.zeros((3, 2, 64), device=DEV)
    pos, f = torch.zeros(3, dtype=torch.int32, device=DEV), freqs(32).to(DEV)
    q.qk_norm_rope(x, k, pos, f)
    w = torch.ones(64, device=DEV)
    for bad in (dict(k=k.to(torch.bfloat16)), dict(k=k[:2]), dict(pos=pos.long()), dict(pos=pos[:2]), dict(f=f.float()),
                dict(f=f.cpu()), dict(q_weight=w[:32]), dict(q_weight=w, k_weight=w.to(torch.bfloat16)),
                dict(q_weight=w.double()), dict(pair_axis=[0] * 31), dict(pos=torch.zeros((2, 3), dtype=torch.int32,
                device=DEV)), dict(x=x.transpose(1, 2)), dict(q_out=x), dict(k_out=k.half()), dict(x=x.half(), k=k.half()),
                dict(q_weight=w.cpu())):
        args = dict(x=x, k=k, pos=pos, f=f)
        args.update({n: bad.pop(n) for n in list(bad) if n in args})
        with pytest.raises(ValueError):
            q.qk_norm_rope(*args.values(), **bad)
    with pytest.raises(q.QGError):
        q.qk_norm_rope(x, k, pos[None].expand(2, 3).contiguous(), f, pair_axis=[2] + [0] * 31)
    with pytest.raises(q.QGError):
        q.qk_norm_rope(x, k, pos, f[:30])


# --------------------------------------------------------------------------
# attention with a shared prefix
# --------------------------------------------------------------------------

def i32(x):
    a = np.asarray(x, dtype=np.int64)
    return torch.from_numpy(a.astype(np.uint32).view(np.int32).copy()).to(DEV)


class Shared:
    """A batch: groups [(prefix length, requests)], `before` and `after` requests without a prefix; lens, nq: own
    tokens and query tokens of all requests in order."""

    def __init__(self, seed, fmt, groups, before, after, lens, nq, Hq, Hkv, D, bs, tree=False, spare_rows=0, q_size=1.5):
        rng = np.random.default_rng(seed)
        self.fmt, self.D = fmt, D
        self.plens, R = [p for p, _ in groups], before + after + sum(n for _, n in groups)
        assert len(lens) == len(nq) == R
        self.lens, self.cu = list(lens), np.concatenate(([0], np.cumsum(nq)))
        self.cu_req = before + np.concatenate(([0], np.cumsum([n for _, n in groups])))
        need = [-(-n // bs) for n in self.plens + self.lens]
        nb = sum(need) + 3
        c = rng.integers(0, 256, (2, nb, Hkv, bs, D), dtype=np.uint8)
        if fmt == "i8":
            c[c == 128] = 7
        else:
            c[(c & 0x7F) == 0x7F] ^= 0x10
        self.k, self.v = c
        self.scales = (rng.random((nb, Hkv, 2)) * 2.0 / float(od.QMAX[FMT[fmt]]) + 1e-4).astype(np.float32)
        ids, at = rng.permutation(nb), 0
        tables = []
        for part in (need[:len(groups)], need[len(groups):]):
            t = np.full((len(part), max(1, max(part)) + 1), -1)
            for r, n in enumerate(part):
                t[r, :n] = ids[at:at + n]
                at += n
            tables.append(t)
        self.ptable, self.table = tables
        T = int(self.cu[-1]) + spare_rows
        # the fill-up of D elements keeps scores of some size
        self.q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * q_size).to(torch.bfloat16)
        self.tree = None
        if tree:
            self.tree = np.zeros(T, np.int64)
            for r in range(R):
                for i in range(nq[r]):
                    p = rng.integers(-1, i) if i else -1
                    t = self.cu[r] + i
                    self.tree[t] = ((self.tree[self.cu[r] + p] if p >= 0 else 0) | 1 << min(i, 31)) & 0xFFFFFFFF

    def args(self):
        cache = [torch.from_numpy(x.copy()).to(DEV).view(DT[self.fmt]) for x in (self.k, self.v)]
        return dict(q=self.q.to(DEV), k_cache=cache[0], v_cache=cache[1], scales=torch.from_numpy(self.scales).to(DEV),
                    prefix_table=i32(self.ptable), prefix_lens=i32(self.plens), cu_req=i32(self.cu_req),
                    block_table=i32(self.table), ctx_lens=i32(self.lens), cu_q=i32(self.cu),
                    tree_mask=None if self.tree is None else i32(self.tree))

    def check(self, out, scale=None, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        ref, mag, qk, n, vmax = od.attention_shared(
            self.q.double().numpy(), self.k, self.v, self.scales, self.ptable, self.plens, self.cu_req, self.table,
            self.lens, self.cu, FMT[self.fmt], scale, self.tree)
        qk, n, vmax = qk[..., None], n[..., None], vmax[..., None]
        tol = 2.0 ** -8 * np.abs(ref) + \
            (2.0 ** -11 + 2 * (self.D + 8) * 2.0 ** -23 * qk + n * 2.0 ** -24 + 2.0 ** -20) * mag + n * 2.0 ** -25 * vmax
        T = int(self.cu[-1])
        rows = np.arange(T) if rows is None else rows
        err = (np.abs(out.double().cpu().numpy() - ref) - tol)[rows]
        assert np.all(err <= 0), (err.max(), np.unravel_index(err.argmax(), err.shape))


SHARED = {
    "one": dict(groups=[(1, 1)], before=0, after=0, lens=[1], nq=[1], Hq=1, Hkv=1, D=128, bs=16),
    "two": dict(groups=[(37, 2)], before=0, after=0, lens=[1, 5], nq=[1, 1], Hq=8, Hkv=2, D=128, bs=16),
    "ends": dict(groups=[(129, 3), (0, 2), (16, 0), (127, 1)], before=1, after=2, lens=[3, 1, 40, 16, 2, 7, 9, 33, 5],
                 nq=[1, 1, 2, 1, 1, 3, 1, 0, 1], Hq=8, Hkv=2, D=128, bs=32),
    "rows129": dict(groups=[(700, 43)], before=0, after=0, lens=[1 + i % 9 for i in range(43)], nq=[1] * 43, Hq=6, Hkv=2,
                    D=128, bs=64),
    "rows300": dict(groups=[(3000, 75), (2000, 70)], before=0, after=0, lens=[1 + i % 40 for i in range(145)],
                    nq=[1] * 145, Hq=4, Hkv=1, D=128, bs=48),
    "long": dict(groups=[(9000, 3)], before=0, after=1, lens=[500, 1, 130, 300], nq=[1, 1, 1, 1], Hq=8, Hkv=2, D=128,
                 bs=128),
    "drafts": dict(groups=[(600, 4), (90, 3)], before=1, after=1, lens=[9, 6, 30, 17, 6, 60, 8, 6, 25], nq=[6] * 9, Hq=16,
                   Hkv=2, D=64, bs=16, tree=True),
    "many drafts": dict(groups=[(300, 3)], before=0, after=0, lens=[40, 33, 64], nq=[40, 32, 33], Hq=4, Hkv=2, D=64, bs=32,
                        tree=True),
    "prompt": dict(groups=[(513, 2)], before=0, after=0, lens=[200, 131], nq=[200, 131], Hq=8, Hkv=2, D=128, bs=64),
    "small heads": dict(groups=[(200, 5)], before=0, after=0, lens=[1, 2, 3, 4, 5], nq=[1] * 5, Hq=10, Hkv=2, D=16, bs=16),
    "heads of 80": dict(groups=[(333, 9)], before=1, after=0, lens=list(range(1, 11)), nq=[1] * 10, Hq=4, Hkv=1, D=80,
                        bs=16),
    "heads of 96": dict(groups=[(1500, 40)], before=0, after=0, lens=[3] * 40, nq=[1] * 40, Hq=8, Hkv=2, D=96, bs=80),
    "heads of 208": dict(groups=[(400, 7)], before=0, after=1, lens=[11] * 8, nq=[1] * 8, Hq=6, Hkv=3, D=208, bs=32),
    "heads of 256": dict(groups=[(1000, 20), (50, 2)], before=0, after=0, lens=[5] * 22, nq=[2] * 22, Hq=4, Hkv=2, D=256,
                         bs=16),
    "many groups": dict(groups=[(10 + 7 * i, 1 + i % 3) for i in range(60)], before=0, after=0, lens=[2] * 120,
                        nq=[1] * 120, Hq=4, Hkv=2, D=64, bs=16),
}


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("name", SHARED)
def test_shared_attention(q, name, fmt):
    b = Shared(len(name), fmt, **SHARED[name])
    a = b.args()
    b.check(q.attn_kv8_shared(**a))
    b.check(q.attn_kv8_shared(**a, softmax_scale=0.5 * b.D ** -0.5), scale=0.5 * b.D ** -0.5)


def test_shared_attention_rows_that_see_nothing(q):
    """No prefix tokens and no own ones, or a tree's word of none: zeros; rows behind the last request stay."""
    b = Shared(1, "i8", [(0, 2), (5, 1)], 1, 0, [0, 0, 3, 0], [1, 1, 2, 1], 4, 2, 128, 16, tree=True, spare_rows=3)
    b.tree[1:4] = 0
    a = b.args()
    out = torch.full((8, 4, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    got = q.attn_kv8_shared(**a, out=out)
    assert got.data_ptr() == out.data_ptr()
    b.check(out[:5].clone() if b.q.shape[0] == 5 else torch.cat((out[:5], torch.zeros((3, 4, 128), device=DEV))))
    assert not out[:2].any() and (out[5:] == 9.0).all()
    # request 2 has one own token before its two drafts, which see it alone; request 3 sees the prefix alone
    assert out[2:5].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_shared_attention_garbage_behind_the_ends(q, D):
    """Slots past a prefix's or a context's end hold NaN codes; one query row is NaN, one infinite, one huge."""
    b = Shared(2, "e4m3", [(100, 6)], 0, 1, [5, 1, 17, 2, 2, 2, 40], [1] * 7, 4, 2, D, 64)
    for row, n in [(b.ptable[0], 100)] + list(zip(b.table, b.lens)):
        blk = row[n // 64] if n % 64 else -1
        if blk >= 0:
            b.k[blk][:, n % 64:] = 0x7F
            b.v[blk][:, n % 64:] = 0xFF
    b.q[1, 0, 3] = float("nan")
    b.q[2, 1, 0] = float("inf")
    b.q[3, 2] *= 1e30
    a = b.args()
    out = q.attn_kv8_shared(**a)
    clean = b.q.clone()
    clean[1, 0, 3] = clean[2, 1, 0] = 0
    clean[3, 2] = 0
    assert out[1, 0].isnan().all() and out[2, 1].isnan().all()
    b.q, full = clean, b.q
    ref = out.clone()
    ref[1, 0], ref[2, 1], ref[3, 2] = 0, 0, 0
    want = q.attn_kv8_shared(**{**a, "q": clean.to(DEV)})
    b.check(want)
    for t in range(7):
        for h in range(4):
            if (t, h) not in ((1, 0), (2, 1), (3, 2)):
                assert torch.equal(out[t, h], want[t, h]), (t, h)


def test_shared_attention_is_attention_over_both(q):
    """A prefix of whole blocks against attn_kv8_paged over the joined block lists, and no groups' requests at all."""
    b = Shared(3, "i8", [(512, 9)], 0, 0, [1 + 3 * i for i in range(9)], [1] * 9, 8, 2, 128, 16)
    a = b.args()
    table = i32(np.concatenate((np.repeat(b.ptable[:, :32], 9, 0), b.table), 1))
    both = q.attn_kv8_paged(a["q"], a["k_cache"], a["v_cache"], a["scales"], table, i32(np.array(b.lens) + 512), a["cu_q"])
    got = q.attn_kv8_shared(**a)
    assert (both.float() - got.float()).abs().max() <= 2.0 ** -6 * both.float().abs().max()
    none = q.attn_kv8_shared(**{**a, "cu_req": i32([9, 9])})
    alone = q.attn_kv8_paged(a["q"], a["k_cache"], a["v_cache"], a["scales"], a["block_table"], a["ctx_lens"], a["cu_q"])
    assert (none.float() - alone.float()).abs().max() <= 2.0 ** -8 * alone.float().abs().max()


def test_shared_attention_strides_streams_and_capture(q):
    b = Shared(4, "e4m3", [(700, 30), (90, 4)], 1, 1, [1 + i for i in range(36)], [1] * 36, 8, 2, 128, 16)
    a = b.args()
    want = q.attn_kv8_shared(**a)
    b.check(want)
    # a slice of a fused row, on a stream of its own
    row = torch.zeros((36, 12 * 128 + 8), dtype=torch.bfloat16, device=DEV)
    row[:, 128:9 * 128] = a["q"].flatten(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q.attn_kv8_shared(**{**a, "q": row[:, 128:9 * 128].unflatten(1, (8, 128))}, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    # two graphs on one stream, replayed on others beside one another and an eager call
    graphs, outs = [], []
    for _ in range(2):
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.attn_kv8_shared(**a, out=out)
        graphs.append(g), outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = q.attn_kv8_shared(**a)
        torch.cuda.synchronize()
        assert torch.equal(eager, want) and torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_shared_attention_workspace(q):
    """A given workspace of which only the counters are zeroed, used by calls of several sizes in turn."""
    batches = [Shared(7 + i, "i8", [(n, r)], 0, 1, [3] * (r + 1), [1] * (r + 1), 8, 2, D, 32)
               for i, (n, r, D) in enumerate(((500, 40, 128), (3000, 2, 128), (70, 5, 256), (900, 33, 64)))]
    size = max(q.workspace_size(q.OP_ATTN_KV8_SHARED, M=8, N=2, K=b.D, T=b.q.shape[0]) for b in batches)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    ws[:4096] = 0
    for _ in range(2):
        for b in batches:
            b.check(q.attn_kv8_shared(**b.args(), workspace=ws))
            assert not ws[:4096].any()


@pytest.mark.parametrize("prefix,requests", [(700, 40), (2500, 3)])
def test_shared_attention_far_blocks(q, prefix, requests):
    """Blocks whose codes begin past 2^32, for either of the prefixes' kernels."""
    n = requests + 1
    b = Shared(12, "i8", [(prefix, requests)], 0, 1, [1 + i for i in range(n)], [1] * n, 8, 2, 128, 64)
    a = b.args()
    want = q.attn_kv8_shared(**a)
    b.check(want)
    nb, per = b.k.shape[1] if b.k.ndim == 5 else b.k.shape[0], 2 * 64 * 128
    far = (1 << 32) // per + 5
    big = {}
    for name in ("k_cache", "v_cache"):
        t = torch.empty((far + nb, 2, 64, 128), dtype=torch.int8, device=DEV)
        t[far:] = a[name]
        big[name] = t
    scales = torch.zeros((far + nb, 2, 2), device=DEV)
    scales[far:] = a["scales"]
    move = lambda t: torch.where(t < 0, t, t + far)  # noqa: E731
    got = q.attn_kv8_shared(**{**a, **big, "scales": scales, "prefix_table": move(a["prefix_table"]),
                               "block_table": move(a["block_table"])})
    assert torch.equal(got, want)


def test_shared_attention_most_groups(q):
    """1024 groups of a request each, every third one without a prefix, every fifth without a query."""
    nq = [0 if i % 5 == 4 else 1 for i in range(1024)]
    b = Shared(13, "e4m3", [(0 if i % 3 == 2 else 1 + i % 150, 1) for i in range(1024)], 0, 0, [1 + i % 20 for i in range(1024)],
               nq, 4, 2, 128, 16)
    b.check(q.attn_kv8_shared(**b.args()))


def test_shared_attention_reports(q):
    """Block ids outside the cache count as unseen; lengths past the table are cut; bounds that do not ascend write nothing."""
    b = Shared(5, "i8", [(300, 5)], 0, 1, [4] * 6, [1] * 6, 4, 2, 128, 16)
    b.ptable[0, 3], b.ptable[0, 7], b.table[2, 0] = -5, 10 ** 6, 10 ** 6
    a = b.args()
    b.check(q.attn_kv8_shared(**a))
    assert q.device_error(clear=True) >> 8 == 6
    b = Shared(5, "i8", [(300, 5)], 0, 1, [4] * 6, [1] * 6, 4, 2, 128, 16)
    b.plens = [10 ** 6]
    for row in b.ptable:
        row[row < 0] = 0
    b.check(q.attn_kv8_shared(**b.args()))
    assert q.device_error(clear=True) == 0x603
    b = Shared(5, "i8", [(300, 2), (40, 3)], 0, 1, [4] * 6, [1] * 6, 4, 2, 128, 16)
    a = b.args()
    for bad in (dict(cu_req=i32([0, 3, 2])), dict(cu_req=i32([-1, 2, 5])), dict(cu_req=i32([0, 2, 7])),
                dict(cu_q=i32([0, 1, 2, 1, 4, 5, 6])), dict(cu_q=i32([0, 1, 2, 3, 4, 5, 7]))):
        out = torch.full((6, 4, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        q.attn_kv8_shared(**{**a, **bad}, out=out)
        assert (out == 9.0).all()
        assert q.device_error(clear=True) == 0x604
    b.check(q.attn_kv8_shared(**a))


def test_shared_attention_refusals(q):
    b = Shared(6, "i8", [(30, 2)], 0, 0, [4] * 2, [1] * 2, 4, 2, 128, 16)
    a = b.args()
    for bad in (dict(q=a["q"].float()), dict(q=a["q"][..., :64]), dict(prefix_table=a["prefix_table"].long()),
                dict(prefix_lens=i32([3, 4])), dict(cu_req=i32([0])), dict(ctx_lens=i32([1])), dict(cu_q=i32([0, 1])),
                dict(tree_mask=i32([1])), dict(out=torch.zeros((2, 4, 128), device=DEV)),
                dict(block_table=a["block_table"][:1]), dict(prefix_lens=a["prefix_lens"].cpu())):
        with pytest.raises(ValueError):
            q.attn_kv8_shared(**{**a, **bad})
    with pytest.raises(q.QGError):
        q.attn_kv8_shared(**a, workspace=torch.zeros(4096, dtype=torch.uint8, device=DEV))
    with pytest.raises(q.QGError):
        q.attn_kv8_shared(**a, softmax_scale=-1.0)


# --------------------------------------------------------------------------
# sampling
# --------------------------------------------------------------------------

EPS = 2.0 ** -22


def check_row(x, u, token, prob, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    order, C, n, i = od.sample(x, u, temperature, top_k, top_p, min_p)
    if i < 0:
        assert token == -1 and prob == 0
        return
    # what may be kept: with top_p a little less or more, where its border is near
    kept = {n}
    if top_p < 1 and temperature > 0:
        kept |= {od.sample(x, u, temperature, top_k, top_p * (1 + f) + g * EPS, min_p)[2] for f, g in ((EPS, 1), (-EPS, -1))}
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    probs = []
    j = int(np.nonzero(order == token)[0][0])
    for n in kept:
        lo, hi = (min(int((C[:n] <= (u + f) * C[n - 1]).sum()), n - 1) for f in (-EPS, EPS))
        if lo <= j <= hi:  # the definition's, or one across borders that are near
            d = min(float(x[token]), 3.5e38) - min(float(x[order[0]]), 3.5e38)
            probs.append(np.exp(d / min(float(temperature), 1e30)) / C[n - 1] if temperature > 0 else 1.0)
    assert probs, (token, order[i], n, len(order))
    assert any(abs(prob - p) <= 2.0 ** -21 * p + 2.0 ** -149 for p in probs), (prob, probs)


def run_rows(q, x, u, passed=None, **settings):
    """x: CPU tensor; settings: per-row lists or None."""
    M = x.shape[0]
    t = {n: None if v is None else torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32, device=DEV)
         for n, v in settings.items()}
    tokens, probs = q.sample_logits(x.to(DEV) if passed is None else passed,
                                    torch.tensor(u, dtype=torch.float32, device=DEV), **t)
    tokens, probs = tokens.cpu().numpy(), probs.double().cpu().numpy()
    rows = x.float().numpy()
    for m in range(M):
        own = {n: (np.float32(v[m]) if n != "top_k" else int(v[m])) for n, v in settings.items() if v is not None}
        check_row(rows[m], float(np.float32(u[m])), int(tokens[m]), float(probs[m]), **own)
    return tokens, probs


def settings_mix(rng, M, V):
    return dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.3, 3.0, 20.0], M).tolist(),
                top_k=rng.choice([0, 1, 5, 50, 400, 1500, V - 1, V, 10 * V], M).tolist(),
                top_p=rng.choice([1.0, 0.9, 0.5, 0.99, 0.0, 1e-6, 2.0], M).tolist(),
                min_p=rng.choice([0.0, 0.0, 0.1, 0.01, 1.0, 3.0], M).tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 100, 1000, 4097, 8192, 8193, 16385, 32771, 50021])
def test_sample(q, V, dtype):
    rng = np.random.default_rng(V)
    M = 40
    x = torch.from_numpy(rng.standard_normal((M, V)) * rng.choice([0.3, 2.0, 6.0], (M, 1))).to(dtype)
    u = rng.random(M).tolist()
    u[0], u[1], u[2], u[3] = 0.0, 1 - 2.0 ** -24, 1.0, float("nan")
    run_rows(q, x, u)
    mix = settings_mix(rng, M, V)
    run_rows(q, x, u, **mix)
    for name in mix:
        run_rows(q, x, u, **{name: mix[name]})
    run_rows(q, x, u, top_k=mix["top_k"], top_p=mix["top_p"])
    d = x.to(DEV), torch.tensor(u, device=DEV)
    long = torch.tensor(mix["top_k"], device=DEV) * (1 << 33)   # above 32 bits: no cut
    for k in (long, long.sign() * 3):
        assert all(map(torch.equal, q.sample_logits(*d, top_k=k), q.sample_logits(*d, top_k=k.clamp(max=1 << 30).int())))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [131075, 151936, 262147, 393216])
def test_sample_large(q, V, dtype):
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((8, V)) * 2).to(dtype)
    x[::2, rng.integers(0, V, 30)] += 9
    u = rng.random(8).tolist()
    run_rows(q, x, u)
    run_rows(q, x, u, temperature=[0.7] * 8, top_k=[50] * 8, top_p=[0.95] * 8)
    run_rows(q, x, u, **settings_mix(rng, 8, V))
    run_rows(q, x, u, temperature=[0.8, 1.0, 1.5, 2.5] * 2, top_p=[0.5, 0.9, 0.99, 0.9999] * 2)


@pytest.mark.parametrize("V", [50, 3000, 20000])
def test_sample_strided_rows(q, V):
    """Rows that begin at any place, of both types."""
    rng = np.random.default_rng(V)
    for dtype in (torch.float32, torch.bfloat16):
        for pad in (1, 2, 3, 5, 7):
            big = torch.full((9, V + pad), float("nan"), dtype=dtype)
            big[:, :V] = torch.from_numpy(rng.standard_normal((9, V)) * 3).to(dtype)
            dev = big.to(DEV)
            run_rows(q, big[:, :V], rng.random(9).tolist(), passed=dev[:, :V], top_p=[0.9] * 9)
            run_rows(q, big[:, :V], rng.random(9).tolist(), passed=dev[:, :V], temperature=[0.0] * 9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(130, 50021), (470, 8195), (240, 20001), (160, 90001)])
def test_sample_many_rows(q, M, V, dtype):
    """More rows than are held at once; rows that begin anywhere; equal logits, masks and numbers that are none among them."""
    rng = np.random.default_rng(M)
    big = torch.full((M, V + 3), float("nan"), dtype=dtype)
    x = big[:, :V]
    x.copy_(torch.from_numpy(rng.standard_normal((M, V)) * rng.choice([0.3, 2.0, 6.0], (M, 1))))
    x[3], x[4], x[5, ::2], x[6, 100:] = 1.5, float("-inf"), float("nan"), float("-inf")
    x[7, 9], x[8], x[9, 5:] = float("inf"), -torch.finfo(dtype).max, 0.25
    clean = x.float().clamp(max=torch.finfo(dtype).max).to(dtype) if dtype == torch.bfloat16 else x
    dev, u = big.to(DEV)[:, :V], rng.random(M).tolist()
    run_rows(q, clean, u, passed=dev)
    run_rows(q, clean, u, passed=dev, **settings_mix(rng, M, V))
    run_rows(q, clean, u, passed=dev, temperature=[0.8] * M, top_p=rng.choice([0.5, 0.9, 0.99], M).tolist())


def test_sample_inverts_the_distribution(q):
    """Evenly spaced numbers give every token its share of them."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal(50)).float()
    M = 4096
    u = ((np.arange(M) + 0.5) / M).tolist()
    tokens, probs = run_rows(q, x.expand(M, 50).contiguous(), u)
    p = torch.softmax(x.double(), 0).numpy()
    counts = np.bincount(tokens, minlength=50)
    assert np.abs(counts - p * M).max() <= 1.0 + 1e-3


@pytest.mark.parametrize("V", [40, 1500, 9000, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_equal_logits(q, V, dtype):
    """All logits equal, or of three values: the lower index comes first, cuts fall among equal ones."""
    rng = np.random.default_rng(V)
    M = 10
    u = rng.random(M).tolist()
    x = torch.full((M, V), 1.5, dtype=dtype)
    run_rows(q, x, u)
    run_rows(q, x, u, top_k=[7, 1, 0, V - 1, V // 2, V // 3, 20, 30, 2, 5])
    run_rows(q, x, u, top_p=[0.5, 0.1, 0.9, 1.0, 0.25, 0.75, 0.3, 0.6, 0.7, 0.8])
    assert run_rows(q, x, u, temperature=[0.0] * M)[0].tolist() == [0] * M
    x = torch.tensor([3.0, 2.0, -0.0, 0.0])[torch.from_numpy(rng.integers(0, 4, (M, V)))].to(dtype)
    run_rows(q, x, u, top_k=[V // 2] * 5 + [V // 5] * 5, top_p=[0.9, 0.5] * 5, min_p=[0.0, 0.2] * 5)
    run_rows(q, x, u, temperature=[2.0] * M)


def test_sample_masks_and_numbers_that_are_none(q):
    rng = np.random.default_rng(2)
    V, inf, nan = 9000, float("inf"), float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        most = torch.finfo(dtype).max
        x = torch.from_numpy(rng.standard_normal((12, V)) * 2).to(dtype)
        x[0] = -inf                                  # nothing to draw
        x[1] = nan
        x[2] = -inf
        x[2, 777] = -5.0                             # one token
        x[3, ::2] = -inf                             # a mask
        x[4, 100:8000] = nan
        x[5, 17] = inf                               # counts as the largest number: drawn
        x[6, [40, 3000]] = inf
        x[7] = -most                                 # a mask of the type's lowest value, everywhere
        x[8] = -most
        x[8, 5:9] = 1.0
        x[9] = most
        x[10, :4000] = -inf
        x[10, 8999] = most
        u = rng.random(12).tolist()
        for setting in (dict(), dict(top_k=[50] * 12), dict(top_p=[0.9] * 12), dict(min_p=[0.1] * 12),
                        dict(temperature=[0.0] * 12), dict(temperature=[1e-38, 1e-20, 0.01, 0.1, 1e9, inf] * 2),
                        dict(temperature=[5.0] * 12, top_k=[20] * 12, top_p=[0.8] * 12)):
            y = x.float().clamp(max=most).to(dtype) if dtype == torch.bfloat16 else x
            tokens, probs = run_rows(q, y, u, passed=x.to(DEV), **setting)
            assert tokens[:2].tolist() == [-1, -1] and tokens[2] == 777 and tokens[5] == 17 and tokens[6] in (40, 3000)
            assert tokens[8] in (5, 6, 7, 8) or (setting.get("temperature") or [0])[0] == 1e-38
    # a temperature that is no number is greedy; negative settings are none
    x = torch.from_numpy(rng.standard_normal((3, 100))).float()
    t, p = q.sample_logits(x.to(DEV), torch.full((3,), 0.7, device=DEV), temperature=torch.tensor([nan, -1.0, -inf], device=DEV))
    assert torch.equal(t.cpu().long(), x.argmax(1)) and (p == 1).all()
    run_rows(q, x, [0.7] * 3, top_k=[-1, -100, 0], min_p=[-1.0, 0.0, -0.5])
    t, _ = q.sample_logits(x.to(DEV), torch.full((3,), 0.7, device=DEV), top_p=torch.full((3,), nan, device=DEV),
                           min_p=torch.full((3,), nan, device=DEV))
    assert torch.equal(t, q.sample_logits(x.to(DEV), torch.full((3,), 0.7, device=DEV))[0])


def test_sample_far_tails(q):
    """Draws and cuts below the bins: a lone head far above a bulk that has most of the mass, cold and hot rows."""
    rng = np.random.default_rng(4)
    V = 30000
    x = torch.from_numpy(rng.standard_normal((8, V))).float()
    x[:, 11] += torch.tensor([20.0, 40.0, 10.0, 25.0, 30.0, 60.0, 100.0, 15.0])
    u = rng.random(8).tolist()
    run_rows(q, x, u, temperature=[5.0, 8.0, 2.0, 6.0, 10.0, 20.0, 30.0, 64.0])
    run_rows(q, x, u, temperature=[5.0, 8.0, 2.0, 6.0, 10.0, 20.0, 30.0, 64.0], top_p=[0.999] * 4 + [0.5] * 4)
    run_rows(q, x, u, temperature=[4.0] * 8, top_k=[300, 3000, 20000, 29999] * 2)
    run_rows(q, x, u, temperature=[0.02] * 8, top_k=[300, 3000] * 4)
    run_rows(q, x, [0.9999999] * 8, temperature=[1.0] * 8)


def test_sample_streams_and_capture(q):
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((20, 60000)) * 2).float()
    d, u = x.to(DEV), torch.rand(20, generator=gen(1)).to(DEV)
    kw = dict(temperature=torch.full((20,), 0.8, device=DEV), top_k=torch.full((20,), 40, dtype=torch.int32, device=DEV))
    want, wp = q.sample_logits(d, u, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    tokens, probs = torch.empty_like(want), torch.empty_like(wp)
    got = q.sample_logits(d, u, **kw, tokens=tokens, probs=probs, stream=s)
    s.synchronize()
    assert torch.equal(tokens, want) and torch.equal(probs, wp) and got[0].data_ptr() == tokens.data_ptr()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = q.sample_logits(d, u, **kw)
    for _ in range(3):
        u.copy_(torch.rand(20, generator=gen(7)).to(DEV))
        g.replay()
        torch.cuda.synchronize()
        e, f = q.sample_logits(d, u, **kw)
        assert torch.equal(a, e) and torch.equal(b, f)


def test_sample_offsets_past_32_bits(q):
    """A row that begins past 2^32 bytes, of the cluster's form and of a CTA's."""
    V = 50021
    for M in (3, 300):
        stride = (1 << 31) // (M - 1) + 7
        whole = torch.empty((M - 1) * stride + V, dtype=torch.bfloat16, device=DEV)
        x = whole.as_strided((M, V), (stride, 1))
        rows = torch.randn((M, V), generator=gen(M)).mul(2).to(torch.bfloat16).to(DEV)
        x.copy_(rows)
        u = torch.rand(M, generator=gen(M + 1)).to(DEV)
        for kw in ({}, dict(top_k=torch.full((M,), 40, dtype=torch.int32, device=DEV))):
            a, b = q.sample_logits(x, u, **kw)
            c, d = q.sample_logits(rows, u, **kw)
            assert torch.equal(a, c) and torch.equal(b, d)


def test_sample_refusals(q):
    x, u = torch.zeros((3, 100), device=DEV), torch.zeros(3, device=DEV)
    for bad in (dict(logits=x.double()), dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.t()), dict(u=u[:2]),
                dict(u=u.double()), dict(u=u.cpu()), dict(temperature=u[:1]), dict(top_k=u), dict(top_p=u.double()),
                dict(min_p=u.int()), dict(tokens=u), dict(probs=u.int())):
        with pytest.raises(ValueError):
            q.sample_logits(**{**dict(logits=x, u=u), **bad})
    with pytest.raises(q.QGError):
        q.sample_logits(torch.zeros((1, 400000), device=DEV), u[:1])
