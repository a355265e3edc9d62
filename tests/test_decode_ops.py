"""CPU side of the decode step's operators: the oracle's pins and the refusals
of malformed requests (no launch happens)."""
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


def test_e4m3_table_and_encoder():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(od.E4M3_VALUES))
    ok = ~np.isnan(v)
    assert np.array_equal(v[ok], od.E4M3_VALUES[ok].astype(np.float32))
    x = torch.cat((torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 60,
                   torch.randn(20000, generator=torch.Generator().manual_seed(2)) * 0.01,
                   torch.tensor([0.0, -0.0, 448.0, -448.0, 447.9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])))
    x = x.clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(od.encode(x.numpy(), od.E4M3), want)


def test_int8_encoder_ties_and_clamp():
    x = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.4, 300.0, -300.0], np.float32)
    assert od.encode(x, od.I8).view(np.int8).tolist() == [0, 2, 2, 0, -2, 126, 127, 127, -127]


def test_append_oracle_by_hand():
    # one block of 16 slots, one head, D = 2: a token at slot 0, then one at slot 1 that doubles the scale
    cache, scales = np.full((1, 1, 16, 2), 9, np.uint8), np.array([[7.0]], np.float32)
    cache, scales = od.append(np.array([[[127.0, -63.4]]]), [0], cache, scales, od.I8, 1, 16)
    assert scales[0, 0] == 1.0 and cache[0, 0, 0].view(np.int8).tolist() == [127, -63]
    assert not cache[0, 0, 1:].any()
    cache, scales = od.append(np.array([[[254.0, 2.0]]]), [1], cache, scales, od.I8, 1, 16)
    assert scales[0, 0] == 2.0
    assert cache[0, 0, :2].view(np.int8).tolist() == [[64, -32], [127, 1]]  # 63.5 -> 64, -31.5 -> -32 (even)
    cache, scales = od.append(np.array([[[3.0, 4.0]]]), [2], cache, scales, od.I8, 1, 16)
    assert scales[0, 0] == 2.0 and cache[0, 0, 2].view(np.int8).tolist() == [2, 2]


def test_plan_oracle_grow_then_shrink_is_the_identity():
    rng = np.random.default_rng(0)
    bs, R, maxb, N = 16, 7, 9, 80
    old = rng.integers(0, 60, R)
    new = old + rng.integers(0, 50, R)
    ids = rng.permutation(N)
    table, at = np.full((R, maxb), -1), 40
    for r in range(R):
        k = -(-old[r] // bs)
        table[r, :k] = ids[at:at + k]
        at += k
    free = ids.copy()
    t1, f1, c1, cu, slots, pos, info = od.block_plan(old, new, table, free, 40, bs, 400)
    assert info[3] == 0 and cu[-1] == (new - old).sum() == info[0]
    used = slots[slots >= 0]
    assert len(set(used.tolist())) == len(used)
    t2, f2, c2, *_ = od.block_plan(new, old, t1, f1, c1, bs, 400)
    assert c2 == 40 and np.array_equal(f2[:40], free[:40])


def test_attention_oracle_single_token_and_uniform():
    # one seen token: its value; equal keys: the mean of the values
    k = np.zeros((2, 1, 16, 16), np.uint8)
    v = (np.arange(2 * 16 * 16) % 100).astype(np.uint8).reshape(2, 1, 16, 16)
    scales = np.full((2, 1, 2), 0.5, np.float32)
    q = np.ones((2, 1, 16))
    out, *_ = od.attention(q, k, v, scales, np.array([[1, 0]]), [2], [0, 2], od.I8, 0.25)
    assert np.allclose(out[0, 0], 0.5 * v[1, 0, 0]) and np.allclose(out[1, 0], 0.25 * (v[1, 0, 0] + v[1, 0, 1].astype(float)))
    # a tree row that sees nothing
    out, _, _, seen, _ = od.attention(q, k, v, scales, np.array([[1, 0]]), [2], [0, 2], od.I8, 0.25, tree=[0, 2])
    assert not out[0].any() and seen[0, 0] == 0 and np.allclose(out[1, 0], 0.5 * v[1, 0, 1])


def test_plan_refusals(L):
    def call(R=2, bs=16, maxb=4, N=8, maxt=8, ptr=A, ws=P(A), wsb=256, null=None):
        a = [P(ptr)] * 9
        if null is not None:
            a[null] = None
        return L.kv8_block_plan(a[0], a[1], R, bs, a[2], maxb, a[3], N, a[4], a[5], a[6], a[7], a[8], maxt, P(ptr), ws,
                                wsb, None)
    for i in range(9):
        assert call(null=i) == 1
    assert call(R=0) == 1 and call(R=4097) == 1 and call(maxb=0) == 1 and call(maxt=0) == 1 and call(N=0) == 1
    for bs in (0, 8, 24, 1040):
        assert call(bs=bs) == 1
    assert call(bs=1024, maxb=1 << 21) == 1 and call(bs=1024, N=1 << 21) == 1
    assert call(ptr=A + 4) == 2
    assert call(ws=None) == 4 and call(wsb=8) == 4


def test_append_and_read_refusals(L):
    def app(dt=0, ks=256, vs=256, T=4, H=2, D=128, bs=16, N=8, fmt=0, ptr=A, null=None):
        a = [P(ptr)] * 6
        if null is not None:
            a[null] = None
        return L.kv8_append(a[0], a[1], dt, ks, vs, a[2], T, H, D, bs, N, fmt, a[3], a[4], a[5], None)
    for i in range(6):
        assert app(null=i) == 1
    for bad in (dict(dt=2), dict(ks=255), dict(vs=128), dict(ks=260), dict(T=0), dict(H=0), dict(D=8), dict(D=272),
                dict(D=40), dict(bs=20), dict(N=0), dict(fmt=2), dict(H=1025, ks=1 << 20, vs=1 << 20)):
        assert app(**bad) == 1, bad
    assert app(ptr=A + 8) == 2

    def read(B=1, H=2, D=128, bs=16, N=8, fmt=0, ptr=A, null=None):
        a = [P(ptr)] * 7
        if null is not None:
            a[null] = None
        return L.kv8_read(a[0], B, H, D, bs, N, fmt, a[1], a[2], a[3], a[4], a[5], a[6], None)
    for i in range(7):
        assert read(null=i) == 1
    for bad in (dict(B=0), dict(D=24), dict(bs=0), dict(fmt=-1)):
        assert read(**bad) == 1, bad
    assert read(ptr=A + 2) == 2


def test_attention_refusals(L):
    ws = L.qg_attn_kv8_workspace_size(8, 2, 128)

    def att(qs=1024, R=2, T=2, Hq=8, Hkv=2, D=128, bs=16, N=8, maxb=4, fmt=0, sc=0.1, ptr=A, w=P(A), wsb=1 << 30,
            null=None, tree=None):
        a = [P(ptr)] * 8
        if null is not None:
            a[null] = None
        return L.attn_kv8_paged(a[0], qs, a[1], a[2], a[3], a[4], a[5], a[6], tree, R, T, Hq, Hkv, D, bs, N, maxb, fmt,
                                sc, a[7], w, wsb, None)
    for i in range(8):
        assert att(null=i) == 1
    for bad in (dict(qs=1016), dict(qs=1028), dict(R=0), dict(R=1025), dict(T=0), dict(Hq=7), dict(Hq=0), dict(Hkv=3),
                dict(D=0), dict(D=264), dict(D=130), dict(bs=8), dict(bs=33), dict(N=0), dict(maxb=0), dict(fmt=3),
                dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=float("inf")),
                dict(bs=1024, maxb=1 << 21), dict(Hq=2050, qs=1 << 20)):
        assert att(**bad) == 1, bad
    assert att(ptr=A + 4) == 2 and att(tree=P(A + 4)) == 2
    if ws:
        assert att(w=None) == 4 and att(wsb=ws - 1) == 4
    assert L.qg_attn_kv8_workspace_size(7, 2, 128) == 0


def test_norm_refusals(L):
    def norm(M=1, K=64, xd=0, rd=0, wd=0, eps=1e-6, x=P(A), res=P(A), w=P(A), ro=P(A), out=P(A)):
        return L.rmsnorm_residual(x, xd, res, rd, w, wd, eps, M, K, ro, out, None)

    def norm8(M=1, K=64, x=P(A), res=P(A), sb=None, ro=P(A), out=P(A), sc=P(A)):
        return L.rmsnorm_residual_i8(x, 0, res, 0, P(A), 0, 1e-6, sb, M, K, ro, out, sc, None)
    for bad in (dict(M=0), dict(K=0), dict(K=48), dict(K=32800), dict(xd=2), dict(rd=-1), dict(wd=5), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(ro=None), dict(out=None)):
        assert norm(**bad) == 1, bad
    for bad in (dict(M=0), dict(K=31), dict(x=None), dict(ro=None), dict(out=None), dict(sc=None)):
        assert norm8(**bad) == 1, bad
    assert norm(x=P(A + 4)) == 2 and norm(out=P(A + 8)) == 2 and norm8(sb=P(A + 4)) == 2 and norm8(sc=P(A + 4)) == 2


def test_device_error_status_names(L):
    assert L.qg_status_string(7).startswith(b"QG_ERR_BAD_INDEX")


def test_workspace_query(L):
    import skinny_gemm_qgemv_gb300 as q
    assert q.workspace_size(q.OP_KV8_PLAN) == L.qg_kv8_plan_workspace_size() > 0
    for D in (16, 64, 80, 128, 256):
        assert q.workspace_size(q.OP_ATTN_KV8, M=8, N=2, K=D) == L.qg_attn_kv8_workspace_size(8, 2, D) > 0
    assert q.workspace_size(q.OP_ATTN_KV8, M=7, N=2, K=128) == 0


def test_attention_workspace_holds_the_widest_pieces(L):
    """The many-row kernel fills heads of up to 128 elements up to 128: its pieces of a split context, 64 rows of 128
    fp32 values with a maximum and a sum each and two of them a CTA, have that size whatever D is."""
    full = L.qg_attn_kv8_workspace_size(8, 2, 128)
    for D in range(16, 129, 16):
        assert L.qg_attn_kv8_workspace_size(8, 2, D) == full, D
    # without a device the query answers for one CTA; a device has more
    assert full >= 4096 + 2 * 64 * (128 * 4 + 8)
    assert L.qg_attn_kv8_workspace_size(8, 2, 256) >= 4096 + 2 * 16 * (256 * 4 + 8)


def test_append_refuses_more_tokens_than_it_counts(L):
    for T in ((1 << 30) + 1, 2 ** 31 - 1):
        assert L.kv8_append(P(A), P(A), 0, 16, 16, P(A), T, 1, 16, 16, 8, 0, P(A), P(A), P(A), None) == 1
