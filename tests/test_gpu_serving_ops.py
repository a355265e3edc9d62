"""GPU parity of the serving step's operators between the projections and the
next token, against their definitions in 64 bits and more.

Tolerances (fixed before the first run):
  * rotation and norm: the sum of squares passes through up to 8 fused steps and
    5 additions, and enters by its square root: r is off by 10 * 2^-24, an
    element of y by 12 * 2^-24; the angle as fp32 half turns by 2^-25 pi, its
    sine and cosine by another 2 units: a pair (u, v) comes out within
    2^-19 (|u| + |v|), and 2^-51 of the whole angle times that; a bf16 result
    within 2^-8 of itself more.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


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
