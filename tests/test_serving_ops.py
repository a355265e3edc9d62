"""CPU side of the serving step's operators between the projections and the next
token: the refusals of malformed requests (no launch happens)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import decode as od

P = ctypes.c_void_p
A = 0x10000  # a fake, 16-byte-aligned "device" address: never dereferenced


@pytest.fixture(scope="module")
def L():
    from skinny_gemm_qgemv_gb300 import build
    import skinny_gemm_qgemv_gb300 as q
    build.build()
    return q.lib()


def test_rope_refusals(L):
    def call(qs=512, ks=256, xd=0, axes=1, rot=64, pair=None, wd=0, eps=1e-6, T=3, Hq=4, Hkv=2, D=128, kd=0, off={}):
        a = {n: P(off.get(n, A)) for n in ("q", "k", "pos", "freq", "qw", "kw", "qo", "ko")}
        return L.qk_norm_rope(a["q"], qs, a["k"], ks, xd, a["pos"], axes, a["freq"], rot, pair, 0, a["qw"], a["kw"], wd,
                              eps, T, Hq, Hkv, D, a["qo"], a["ko"], kd, None)
    for n in ("q", "k", "pos", "freq", "qo", "ko"):
        assert call(off={n: None}) == 1, n
    for n in ("q", "k", "pos", "freq", "qw", "kw", "qo", "ko"):
        assert call(off={n: A + 8}) == 2, n
    for bad in (dict(xd=2), dict(wd=-1), dict(kd=3), dict(T=0), dict(T=(1 << 30) + 1), dict(Hq=0), dict(Hkv=0),
                dict(Hq=1025, qs=1 << 20), dict(Hkv=1025, ks=1 << 20), dict(D=8), dict(D=120, rot=8), dict(D=272),
                dict(rot=0), dict(rot=12), dict(rot=136), dict(qs=511), dict(qs=516), dict(ks=248), dict(axes=0),
                dict(axes=5, pair=bytes(32)), dict(axes=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(axes=2, pair=bytes([2] + [0] * 31)), dict(axes=1, pair=bytes([0] * 31 + [1]))):
        assert call(**bad) == 1, bad


def test_shared_attention_oracle_is_attention_over_both():
    """A prefix of whole blocks: the same as one block list, prefix first; a prefix of none: the requests' own."""
    rng = np.random.default_rng(0)
    nb, Hkv, bs, D, Hq = 12, 2, 16, 16, 4
    k, v = rng.integers(0, 127, (2, nb, Hkv, bs, D), dtype=np.uint8)
    sc = rng.random((nb, Hkv, 2)).astype(np.float32) / 64
    q = rng.standard_normal((5, Hq, D))
    table, ptable = np.array([[0, 1], [2, 3], [4, 5]]), np.array([[6, 7, 8]])
    lens, cu = [17, 5, 30], [0, 2, 4, 5]
    for tree in (None, [1, 2, 1, 3, 1]):
        got = od.attention_shared(q, k, v, sc, ptable, [48], [1, 3], table, lens, cu, od.I8, 0.25, tree)
        both = np.concatenate((np.repeat(ptable, 3, 0), table), 1)
        want = od.attention(q, k, v, sc, both, [65, 53, 78], cu, od.I8, 0.25, tree)
        alone = od.attention(q, k, v, sc, table, lens, cu, od.I8, 0.25, tree)
        for g, w, x in zip(got, want, alone):
            assert np.allclose(g[2:], w[2:]) and np.allclose(g[:2], x[:2])


def test_shared_attention_refusals(L):
    names = ("q", "k", "v", "sc", "pt", "pl", "cr", "bt", "cl", "cu", "tm", "out", "ws")
    need = L.qg_attn_kv8_shared_workspace_size(5, 4, 2, 128)
    assert need > L.qg_attn_kv8_workspace_size(4, 2, 128) > 0
    assert L.qg_workspace_size(8, 4, 2, 128, 5, 0, 0) == need
    for bad in ((0, 4, 2, 128), (5, 5, 2, 128), (5, 4, 2, 24), (1 << 30, 4, 2, 128)):
        assert L.qg_attn_kv8_shared_workspace_size(*bad) == 0

    def call(qs=512, groups=1, R=2, T=5, Hq=4, Hkv=2, D=128, bs=16, nb=8, mpb=4, mb=4, fmt=0, scale=0.1, wsb=need, off={}):
        a = {n: P(off.get(n, A)) for n in names}
        return L.attn_kv8_shared(a["q"], qs, a["k"], a["v"], a["sc"], a["pt"], a["pl"], a["cr"], a["bt"], a["cl"],
                                 a["cu"], a["tm"], groups, R, T, Hq, Hkv, D, bs, nb, mpb, mb, fmt, scale, a["out"],
                                 a["ws"], wsb, None)
    for n in names:
        if n not in ("tm", "ws"):
            assert call(off={n: None}) == 1, n
        assert call(off={n: A + 4}) == 2, n
    for bad in (dict(qs=504), dict(qs=516), dict(groups=0), dict(groups=1025), dict(R=0), dict(R=1025), dict(T=0),
                dict(Hq=5), dict(Hq=0), dict(Hkv=0), dict(D=24), dict(D=272), dict(bs=8), dict(bs=1040), dict(nb=0),
                dict(mpb=0), dict(mb=0), dict(mpb=1 << 28), dict(mb=1 << 28), dict(fmt=2), dict(scale=0.0),
                dict(scale=float("nan"))):
        assert call(**bad) == 1, bad
    assert call(wsb=need - 1) == 4 and call(off=dict(ws=None)) == 4
    assert call(R=1024, T=1 << 20, mb=1 << 26, wsb=1 << 40) == 3
    assert call(groups=1024, T=1 << 20, mpb=1 << 26, wsb=1 << 40) == 3


def test_sample_oracle_by_hand():
    x = np.log([0.1, 0.4, 0.1, 0.2, 0.2])
    for u, want in ((0.0, 1), (0.39, 1), (0.41, 3), (0.59, 3), (0.61, 4), (0.81, 0), (0.91, 2), (0.9999, 2)):
        order, C, n, i = od.sample(x, u)
        assert order.tolist() == [1, 3, 4, 0, 2] and n == 5 and order[i] == want
    assert od.sample(x, 0.99, top_k=2)[2] == 2 and od.sample(x, 0.99, top_p=0.61)[2] == 3
    assert od.sample(x, 0.99, top_k=3, top_p=0.7)[2] == 2          # 0.6 of 0.8 is 0.75
    assert od.sample(x, 0.99, min_p=0.4)[2] == 3 and od.sample(x, 0.99, top_p=0.0)[2] == 1
    assert od.sample(x, 0.99, temperature=0.0)[2:] == (1, 0)
    assert od.sample(np.full(3, -np.inf), 0.5)[3] == -1
    order, _, n, i = od.sample(np.array([np.nan, 1.0, np.inf, np.inf, -np.inf]), 0.6)
    assert order.tolist() == [2, 3, 1] and order[i] == 3


def test_sample_refusals(L):
    names = ("x", "u", "t", "k", "p", "mp", "tok", "pr")

    def call(dt=1, stride=100, M=2, V=100, kb=4, off={}):
        a = {n: P(off.get(n, A)) for n in names}
        return L.sample_logits(a["x"], dt, stride, M, V, a["u"], a["t"], a["k"], kb, a["p"], a["mp"], a["tok"], a["pr"], None)
    for n in names:
        assert call(off={n: A + 8}) == 2, n
    for n in ("x", "u", "tok"):
        assert call(off={n: None}) == 1, n
    for bad in (dict(dt=2), dict(stride=99), dict(M=0), dict(M=(1 << 20) + 1), dict(V=0), dict(kb=2)):
        assert call(**bad) == 1, bad
    assert call(V=393217, stride=393217) == 3


def test_rope_pair_axis_is_a_sequence():
    """A number alone is no list of axes; arrays of any whole type are."""
    import skinny_gemm_qgemv_gb300 as q
    x, pos, f = torch.zeros((3, 4, 64)), torch.zeros((2, 3), dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(TypeError):
        q.qk_norm_rope(x, x, pos, f, pair_axis=32)
    for axes in (np.zeros(32, np.int64), torch.zeros(32, dtype=torch.int64), [0] * 32):
        with pytest.raises(ValueError, match="CUDA|cuda|device"):  # (as far as the tensors' place)
            q.qk_norm_rope(x, x, pos, f, pair_axis=axes)
