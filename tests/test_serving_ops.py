"""CPU side of the serving step's operators between the projections and the next
token: the refusals of malformed requests (no launch happens)."""
import ctypes

import pytest

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
