"""GPU parity of the decode step's operators against the 64-bit oracle.

Tolerances (fixed before the first run):
  * block plan, cache codes and scales, read-back values: equal, bit for bit.
  * attention: |o - ref| <= 2^-8 |ref| (the bf16 result) + (2^-11 + 2 d +
    n 2^-24) sum p|v| + n 2^-25 max|v|, n the seen tokens: the probabilities'
    fp16 rounding, the scores' fp32 error d = (D + 8) 2^-23 max sum|q k| in
    both numerator and denominator, the fp32 sums, and probabilities below
    fp16's normal range.
  * norm: bf16 2^-8 |ref| + 2^-18 |ref| (fp32 sums and products); int8: the
    scale and the codes' values off by e = 48 * 2^-24 sum|y| of the value's
    32-block (or of |y|), the code by half a step more; a row's scale
    additionally by that error of its largest value.
"""
import math

import numpy as np
import pytest
import torch

import synth
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


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.uint32).view(np.int32) if np.asarray(x).size else
                        np.zeros(0, np.int32), device=DEV)


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


# --------------------------------------------------------------------------
# block plan
# --------------------------------------------------------------------------

def plan_state(rng, R, bs, top, grow, spare):
    old = rng.integers(0, top + 1, R)
    new = np.where(rng.random(R) < 0.2, rng.integers(0, old + 1), old + rng.integers(0, grow + 1, R))
    have, need = -(-old // bs), -(-new // bs)
    free = int(np.maximum(need - have, 0).sum()) + spare
    N, maxb = free + int(have.sum()), int(max(have.max(), need.max(), 1))
    ids = rng.permutation(N).astype(np.int32)
    table, at = np.full((R, maxb), -7, np.int32), free
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    return old, new, table, ids, free


def run_plan(q, old, new, table, free, count, bs, max_tokens, inplace=False):
    t, f, c = i32(table), i32(free), i32([count])
    got = q.kv8_block_plan(i32(old), i32(new), t, f, c, bs, max_tokens, free_count_out=c if inplace else None)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, f, *got)], (t, f, got[0])


@pytest.mark.parametrize("R,bs,top,grow", [(1, 16, 0, 1), (1, 64, 100, 5000), (3, 16, 40, 1), (32, 16, 500, 1),
                                           (33, 48, 100, 70), (513, 32, 90, 33), (1000, 1024, 5000, 3000),
                                           (4096, 16, 40, 9)])
@pytest.mark.parametrize("inplace", [False, True])
def test_plan(q, R, bs, top, grow, inplace):
    rng = np.random.default_rng(R + bs)
    old, new, table, free, count = plan_state(rng, R, bs, top, grow, 3)
    tokens = int(np.maximum(new - old, 0).sum())
    for max_tokens in {max(1, tokens), tokens + 1 + R % 7}:
        got, dev = run_plan(q, old, new, table, free, count, bs, max_tokens, inplace)
        want = od.block_plan(old, new, table, free, count, bs, max_tokens)
        for g, w, name in zip(got, want, ("table", "free_list", "count", "cu", "slots", "positions", "info")):
            assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name
        assert want[-1][3] == 0
    # back again: the stack below the count is what it was
    t, f, c = dev
    back = q.kv8_block_plan(i32(new), i32(old), t, f, c, bs, max(1, int(np.maximum(old - new, 0).sum())))
    want = od.block_plan(new, old, *[x for x in want[:3]], bs, max(1, int(np.maximum(old - new, 0).sum())))
    torch.cuda.synchronize()
    assert back[4][3].item() == 0 and back[0].item() == count
    assert np.array_equal(f.cpu().numpy(), want[1])


def test_plan_states(q):
    rng = np.random.default_rng(9)
    old, new, table, free, count = plan_state(rng, 20, 16, 100, 40, 0)
    tokens = int(np.maximum(new - old, 0).sum())
    grown = np.maximum(old, new)
    cases = [(old, grown, 0, tokens, 1), (old, new + 100000, count, tokens, 2), (old, new, count, tokens - 1, 3),
             (old, np.where(np.arange(20) == 7, -1, new), count, tokens, 4), (old, new, -1, tokens, 4),
             (old, new, len(free) + 1, tokens, 4), (old, np.zeros(20, int), len(free), tokens, 4),
             (old, np.full(20, 2 ** 31 - 1), count, tokens, 2)]
    for o, n, c, mt, state in cases:
        got, _ = run_plan(q, o, n, table, free, c, 16, mt)
        want = od.block_plan(o, n, table, free, c, 16, mt)
        assert got[-1].tolist() == [0, 0, 0, state] == want[-1].tolist()
        for g, w in zip(got, want):
            assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), state


# --------------------------------------------------------------------------
# cache
# --------------------------------------------------------------------------

def random_cache(rng, nb, H, bs, D, fmt, device=DEV):
    """Random codes (every int8 code but -128, every finite e4m3 code) and scales."""
    c = rng.integers(0, 256, (2, nb, H, bs, D), dtype=np.uint8)
    if fmt == "i8":
        c[c == 128] = 7
    else:
        c[(c & 0x7F) == 0x7F] ^= 0x10
    scales = (rng.random((nb, H, 2)) * 2.0 / float(od.QMAX[FMT[fmt]]) + 1e-4).astype(np.float32)
    return c[0], c[1], scales


def to_cache(c, fmt):
    return torch.from_numpy(c.copy()).to(DEV).view(DT[fmt])


def check_append(q, fmt, dtype, k, v, slots, kc, vc, sc, nb, bs, kt=None, vt=None):
    """k, v: fp32 tensors (already rounded to dtype); kt, vt: what is passed."""
    kd, vd, sd = to_cache(kc, fmt), to_cache(vc, fmt), torch.from_numpy(sc.copy()).to(DEV)
    q.kv8_append(k.to(dtype).to(DEV) if kt is None else kt, v.to(dtype).to(DEV) if vt is None else vt, i32(slots), kd,
                 vd, sd)
    torch.cuda.synchronize()
    wk, s0 = od.append(k.numpy(), slots, kc, sc[..., 0], FMT[fmt], nb, bs)
    wv, s1 = od.append(v.numpy(), slots, vc, sc[..., 1], FMT[fmt], nb, bs)
    assert np.array_equal(sd.cpu().numpy(), np.stack((s0, s1), -1))
    assert np.array_equal(bits(kd), wk) and np.array_equal(bits(vd), wv)
    return kd, vd, sd, wk, wv, np.stack((s0, s1), -1)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs,runs", [
    (1, 16, 16, [(0, 1)]), (2, 64, 16, [(3, 5), (0, 16), (15, 1)]), (8, 128, 16, [(i % 16, 1) for i in range(32)]),
    (3, 80, 48, [(0, 48), (0, 48), (0, 7)]), (1, 256, 64, [(1, 63), (0, 64)]), (2, 128, 256, [(0, 200), (31, 225)]),
    (2, 64, 1024, [(1000, 24), (0, 1024)]), (1, 128, 32, [(31, 1), (0, 31)])])
def test_append(q, fmt, dtype, H, D, bs, runs):
    rng = np.random.default_rng(H * D + bs)
    nb = len(runs) + 2
    kc, vc, sc = random_cache(rng, nb, H, bs, D, fmt)
    blocks = rng.permutation(nb)[:len(runs)]
    slots = np.concatenate([b * bs + f + np.arange(n) for b, (f, n) in zip(blocks, runs)])
    T = len(slots)
    g = torch.Generator().manual_seed(T)
    # some tokens raise their block's scale, some do not, some are zero
    size = torch.tensor([0.0, 0.01, 1.0, 30.0])[torch.randint(0, 4, (T, 1, 1), generator=g)]
    k, v = ((torch.randn((T, H, D), generator=g) * size).to(dtype).float() for _ in range(2))
    kd, vd, sd, wk, wv, ws = check_append(q, fmt, dtype, k, v, slots, kc, vc, sc, nb, bs)
    ids = rng.permutation(nb)
    rk, rv, rs = q.kv8_read(i32(ids), kd, vd, sd)
    torch.cuda.synchronize()
    assert np.array_equal(rs.cpu().numpy(), ws[ids])
    for got, w, which in ((rk, wk, 0), (rv, wv, 1)):
        want = (torch.from_numpy(od.decode(w[ids], FMT[fmt]).astype(np.float32)) *
                torch.from_numpy(ws[ids][..., which])[..., None, None]).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_steps_fill_a_block(q, fmt):
    """Sixteen one-token appends into one block, each step checked: the scale grows and the codes are rounded again."""
    rng = np.random.default_rng(3)
    kc, vc, sc = random_cache(rng, 3, 2, 16, 64, fmt)
    g = torch.Generator().manual_seed(4)
    for s in range(16):
        k, v = (torch.randn((1, 2, 64), generator=g) * (1 + 0.5 * s) for _ in range(2))
        _, _, _, kc, vc, sc = check_append(q, fmt, torch.float32, k, v, [16 + s], kc, vc, sc, 3, 16)


def test_append_strided_padded_and_zero(q):
    rng = np.random.default_rng(5)
    H, D, bs, nb, T = 4, 64, 16, 6, 23
    kc, vc, sc = random_cache(rng, nb, H, bs, D, "i8")
    # slices of a fused q/k/v row; padding slots before, between and after the runs
    fused = torch.randn((T, 3 * H * D + 8), generator=torch.Generator().manual_seed(6))
    fused[5:9] = 0
    fd = fused.to(DEV)
    kt = fd[:, H * D:2 * H * D].unflatten(1, (H, D))
    vt = fd[:, 2 * H * D:3 * H * D].unflatten(1, (H, D))
    slots = np.array([-1, -1] + list(range(80, 88)) + [-1] + list(range(32, 42)) + [-5, -1])
    check_append(q, "i8", torch.float32, kt.cpu().contiguous(), vt.cpu().contiguous(), slots, kc, vc, sc, nb, bs, kt, vt)
    # a new block of zeros: scale 0, codes 0
    z = torch.zeros((16, H, D))
    _, _, sd, wk, _, ws = check_append(q, "i8", torch.float32, z, z, np.arange(16), kc, vc, sc, nb, bs)
    assert not ws[0].any() and not wk[0].any()


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("ulps", [1, 100, 178, 700, 5000, 200000])
def test_append_subnormal_scales(q, fmt, ulps):
    """Values of some 2^-149: the scale is subnormal, so a quotient can pass qmax and is clamped there."""
    rng = np.random.default_rng(ulps)
    kc, vc, sc = random_cache(rng, 2, 2, 16, 64, fmt)
    g = torch.Generator().manual_seed(ulps)
    k, v = ((torch.randint(-ulps, ulps + 1, (16, 2, 64), generator=g).double() * 2.0 ** -149).float() for _ in range(2))
    k[3, :, 5], v[4, :, 7] = ulps * 2.0 ** -149, -ulps * 2.0 ** -149
    check_append(q, fmt, torch.float32, k, v, 16 + np.arange(16), kc, vc, sc, 2, 16)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_largest_values(q, fmt):
    rng = np.random.default_rng(2)
    kc, vc, sc = random_cache(rng, 2, 2, 16, 64, fmt)
    top = torch.finfo(torch.float32).max
    k = torch.rand((16, 2, 64), generator=torch.Generator().manual_seed(1)) * 2 - 1
    k = k * top
    k[2, :, 3] = top
    check_append(q, fmt, torch.float32, k, -k, np.arange(16), kc, vc, sc, 2, 16)


def test_bad_slots_and_blocks_are_skipped_and_reported(q):
    rng = np.random.default_rng(7)
    kc, vc, sc = random_cache(rng, 4, 2, 16, 64, "i8")
    k = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(8))
    check_append(q, "i8", torch.float32, k, k, [64, 5, 2 ** 31 - 1], kc, vc, sc, 4, 16)
    assert q.device_error(clear=True) == 0x601
    rk, rv, rs = q.kv8_read(i32([4, 1, 2 ** 32 - 1]), to_cache(kc, "i8"), to_cache(vc, "i8"), torch.from_numpy(sc).to(DEV))
    torch.cuda.synchronize()
    assert not rk[0].any() and not rv[2].any() and not rs[0].any() and rk[1].any()
    assert q.lib().qg_device_error(None, 1) == 7


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

def attn_case(rng, nq, ctx, Hq, Hkv, D, bs, fmt, tree, qstd=1.0):
    R = len(nq)
    need = [-(-max(c, 0) // bs) for c in ctx]
    nb, maxb = sum(need) + 2, max(max(need), 1)
    kc, vc, sc = random_cache(rng, nb, Hkv, bs, D, fmt)
    ids = rng.permutation(nb)
    table, at = np.full((R, maxb), -1, np.int64), 0
    for r in range(R):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        if need[r] and ctx[r] % bs:
            # slots past the context: anything, also codes that are not numbers
            for c in (kc, vc):
                c[table[r, need[r] - 1], :, ctx[r] % bs:] = 0x7F if fmt == "e4m3" else 0x80
    cu = np.concatenate(([0], np.cumsum(nq)))
    T = int(cu[-1]) + 3                                  # rows past the last request stay as they are
    x = (torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(int(rng.integers(1 << 30)))) * qstd).to(
        torch.bfloat16)
    masks = None
    if tree:
        masks = np.zeros(T, np.int64)
        for r in range(R):
            for i in range(nq[r]):
                parent = int(rng.integers(-1, i)) if i else -1
                masks[cu[r] + i] = (masks[cu[r] + parent] if parent >= 0 else 0) | (1 << (i % 32))
    return dict(x=x, kc=kc, vc=vc, sc=sc, table=table, ctx=np.asarray(ctx), cu=cu, masks=masks, fmt=fmt)


def run_attn(q, c, x=None, **kw):
    out = torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16)
    q.attn_kv8_paged(c["x"].to(DEV) if x is None else x, to_cache(c["kc"], c["fmt"]), to_cache(c["vc"], c["fmt"]),
                     torch.from_numpy(c["sc"]).to(DEV), i32(c["table"]), i32(c["ctx"]), i32(c["cu"]),
                     tree_mask=None if c["masks"] is None else i32(c["masks"]), out=out, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def check_attn(out, c, scale=None):
    D = c["x"].shape[2]
    ref, mag, qk, n, vmax = od.attention(c["x"].float().numpy(), c["kc"], c["vc"], c["sc"], c["table"], c["ctx"],
                                         c["cu"], FMT[c["fmt"]], D ** -0.5 if scale is None else scale, c["masks"])
    last = int(c["cu"][-1])
    assert bool((out[last:] == 7.0).all())
    o = out[:last].double().numpy()
    assert np.isfinite(o).all()
    ref, mag, qk, n, vmax = ref[:last], mag[:last], qk[:last, :, None], n[:last, :, None], vmax[:last, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * qk + n * 2.0 ** -24) * mag + \
        n * 2.0 ** -25 * vmax
    bad = np.abs(o - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}; worst {np.max(np.abs(o - ref) / np.maximum(tol, 1e-300)):.3g}x"
    assert not o[np.broadcast_to(n == 0, o.shape)].any()


CASES = [
    # query tokens, context lengths, Hq, Hkv, D, block, tree
    ([1], [1], 4, 1, 128, 16, False),
    ([1], [37], 32, 8, 128, 16, False),
    ([1], [700], 8, 8, 128, 64, False),
    ([1, 1, 1, 1, 1], [1, 16, 17, 0, 1000], 8, 2, 128, 16, False),
    ([1, 0, 3, 2, 1], [50, 90, 3, 1, 333], 10, 2, 64, 32, False),
    ([1] * 33, [(i * 97) % 400 for i in range(33)], 6, 2, 64, 16, False),
    ([4, 5, 1], [129, 64, 80], 16, 2, 128, 48, False),
    ([16], [2063], 32, 8, 128, 64, True),
    ([16, 1, 32, 7], [16, 1, 32, 200], 8, 2, 128, 16, True),
    ([32], [515], 7, 1, 64, 32, True),
    ([40, 33], [40, 300], 4, 2, 128, 16, True),
    ([100], [1000], 4, 1, 128, 128, False),
    ([1, 2], [300, 45], 8, 2, 256, 16, False),
    ([16, 3], [90, 600], 8, 1, 256, 64, True),
    ([1, 6], [77, 140], 6, 3, 80, 16, False),
    ([5], [64], 4, 4, 16, 16, True),
    ([1], [5000], 5, 1, 64, 1024, False),
    ([1, 1], [70, 40], 64, 2, 128, 16, False),
    ([2], [260], 48, 1, 64, 48, False),
]


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("nq,ctx,Hq,Hkv,D,bs,tree", CASES)
def test_attention(q, fmt, nq, ctx, Hq, Hkv, D, bs, tree):
    rng = np.random.default_rng(sum(ctx) + D + Hq)
    c = attn_case(rng, nq, ctx, Hq, Hkv, D, bs, fmt, tree)
    out = run_attn(q, c)
    check_attn(out, c)
    assert torch.equal(run_attn(q, c), out)  # the same bits again


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [16, 48, 96, 112, 144, 192, 240])
@pytest.mark.parametrize("nq", [1, 5])
def test_attention_head_sizes(q, fmt, D, nq):
    """Heads between the widths that the kernels are made for, alone in a split context and in a ragged batch."""
    rng = np.random.default_rng(D + nq)
    for R, ctx in (([nq], [4000]), ([nq, nq, 1], [nq, 333, 61])):
        c = attn_case(rng, R, ctx, 6, 2, D, 32, fmt, nq > 1)
        check_attn(run_attn(q, c), c)


def test_attention_masks_that_leave_nothing(q):
    # drafts without any earlier token, their words empty or naming tokens past the drafts
    rng = np.random.default_rng(21)
    c = attn_case(rng, [4, 3], [4, 3], 8, 2, 128, 16, "i8", True)
    c["masks"][:] = [0, 0b1, 0, 0xFFFFFFF0, 0b111, 0, 0x80000000, 0, 0, 0]
    out = run_attn(q, c)
    check_attn(out, c)
    assert not out[0].any() and not out[2].any() and not out[5].any() and not out[6].any() and out[1].any()
    # a context shorter than the query tokens: the first ones see nothing
    c = attn_case(rng, [6], [2], 8, 2, 128, 16, "e4m3", False)
    out = run_attn(q, c)
    check_attn(out, c)
    assert not out[:4].any() and out[4].any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_attention_scales_of_all_sizes(q, D, fmt):
    """Blocks of zero scale, and scales that differ by 2^30; large and tiny queries."""
    rng = np.random.default_rng(22)
    c = attn_case(rng, [1, 4], [400, 333], 8, 2, D, 16, fmt, False)
    c["sc"][::3, :, 1] = 0.0
    c["sc"][1::3, :, 1] *= np.float32(2.0 ** -30)
    c["sc"][::5, :, 0] = 0.0
    c["x"][1] *= 1e-6
    c["x"][2] *= 40.0
    check_attn(run_attn(q, c), c)
    c["sc"][..., 1] = 0.0
    assert not run_attn(q, c)[:5].any()
    c["sc"][..., 1] = np.float32(2.0 ** 40)
    check_attn(run_attn(q, c), c)


def test_attention_peaked_scores_and_softmax_scale(q):
    rng = np.random.default_rng(23)
    c = attn_case(rng, [3], [900], 8, 2, 128, 32, "i8", False, qstd=30.0)
    check_attn(run_attn(q, c), c)
    check_attn(run_attn(q, c, softmax_scale=1.7), c, 1.7)
    check_attn(run_attn(q, c, softmax_scale=1e-6), c, 1e-6)


def test_attention_strided_queries(q):
    rng = np.random.default_rng(24)
    c = attn_case(rng, [2, 1], [30, 99], 8, 2, 64, 16, "i8", False)
    T = c["x"].shape[0]
    fused = torch.zeros((T, 12 * 64), dtype=torch.bfloat16, device=DEV)
    fused[:, 128:128 + 8 * 64] = c["x"].reshape(T, -1).to(DEV)
    check_attn(run_attn(q, c, x=fused[:, 128:128 + 8 * 64].unflatten(1, (8, 64))), c)


@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_attention_bad_blocks_and_lengths(q, D):
    rng = np.random.default_rng(25)
    c = attn_case(rng, [1, 2], [200, 90], 4, 2, D, 16, "i8", False)
    c["table"][0, 3], c["table"][0, 7], c["table"][1, 0] = -1, c["kc"].shape[0], 2 ** 31 - 1
    out = run_attn(q, c)
    check_attn(out, c)
    assert q.device_error(clear=True) == 0x602
    c["table"][0, 3], c["table"][0, 7], c["table"][1, 0] = 0, 1, 2
    c["ctx"][0] = 10 ** 6                                # past its table: cut there
    out = run_attn(q, c)
    check_attn(out, c)
    assert q.device_error(clear=True) == 0x603
    assert q.lib().qg_device_error(None, 1) == 0


def test_attention_long_context(q):
    rng = np.random.default_rng(26)
    c = attn_case(rng, [1], [70001], 4, 1, 128, 64, "i8", False)
    check_attn(run_attn(q, c), c)


def test_attention_offsets_past_32_bits(q):
    """A cache of more than 2^32 bytes, its far end used."""
    bs, D, Hkv = 64, 128, 2
    nb = (1 << 32) // (Hkv * bs * D) + 9
    kd = torch.zeros((nb, Hkv, bs, D), device=DEV, dtype=torch.int8)
    vd = torch.zeros((nb, Hkv, bs, D), device=DEV, dtype=torch.int8)
    sd = torch.full((nb, Hkv, 2), 0.01, device=DEV)
    rng = np.random.default_rng(27)
    c = attn_case(rng, [1, 2], [300, 100], 8, Hkv, D, bs, "i8", False)
    small = c["kc"].shape[0]
    kd[nb - small:] = to_cache(c["kc"], "i8")
    vd[nb - small:] = to_cache(c["vc"], "i8")
    sd[nb - small:] = torch.from_numpy(c["sc"]).to(DEV)
    table = np.where(c["table"] >= 0, c["table"] + nb - small, -1)
    out = torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16)
    q.attn_kv8_paged(c["x"].to(DEV), kd, vd, sd, i32(table), i32(c["ctx"]), i32(c["cu"]), out=out)
    check_attn(out.cpu(), c)
    # and an append and a read there
    k = torch.randn((2, Hkv, D), generator=torch.Generator().manual_seed(1))
    slots = [(nb - 1) * bs, (nb - 1) * bs + 1]
    q.kv8_append(k.to(DEV), k.to(DEV), i32(slots), kd, vd, sd)
    rk, rv, rs = q.kv8_read(i32([nb - 1]), kd, vd, sd)
    assert torch.equal(rk, rv)
    scale = k.abs().amax((0, 2)) / 127
    assert torch.equal(rs[0, :, 0].cpu(), scale)
    assert bool(((rk[0, :, :2].float().cpu().transpose(0, 1) - k).abs() <= scale[:, None] * 0.51 + 2.0 ** -8 * k.abs()
                 ).all())


def test_outputs_belong_to_the_given_stream(q):
    """An output made for another stream does not take memory that the current stream still uses."""
    s = torch.cuda.Stream()
    x, w = torch.randn((64, 4096), device=DEV), torch.ones(4096, device=DEV)
    want, _ = q.rmsnorm_residual(x, w)
    torch.cuda.synchronize()
    big = torch.randn((4096, 4096), device=DEV)
    for _ in range(4):
        old = torch.empty((64, 4096), device=DEV, dtype=torch.bfloat16)
        for _ in range(6):
            big @ big                                    # the current stream is busy
        old.fill_(3.0)                                   # written late
        del old                                          # and given back to the current stream's pool
        got, _ = q.rmsnorm_residual(x, w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_attention_on_another_stream_and_in_a_graph(q):
    rng = np.random.default_rng(28)
    c = attn_case(rng, [1, 2, 1], [100, 400, 37], 8, 2, 128, 16, "i8", False)
    want = run_attn(q, c)
    dev = [c["x"].to(DEV), to_cache(c["kc"], "i8"), to_cache(c["vc"], "i8"), torch.from_numpy(c["sc"]).to(DEV),
           i32(c["table"]), i32(c["ctx"]), i32(c["cu"])]
    out = torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q.attn_kv8_paged(*dev, out=out)
    st.synchronize()
    assert torch.equal(out.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_kv8_paged(*dev, out=out)
    # the lengths and tables are read by the replay
    dev[5].copy_(i32([64, 5, 37]))
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    c["ctx"] = np.array([64, 5, 37])
    check_attn(out.cpu(), c)


def test_decode_ops_back_to_back_with_pdl(q):
    """plan -> append -> attention on one stream, launched with programmatic dependent launch: the same bits."""
    rng = np.random.default_rng(29)
    R, bs, Hkv, D = 5, 16, 2, 128
    old = np.array([0, 15, 16, 33, 200])
    new = old + np.array([3, 1, 1, 4, 2])
    need = -(-old // bs)
    nb, maxb = int(need.sum()) + 9, 14
    ids = rng.permutation(nb)
    table = np.full((R, maxb), -1)
    at = 9
    for r in range(R):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    kc, vc, sc = random_cache(rng, nb, Hkv, bs, D, "e4m3")
    T = int((new - old).sum())
    g = torch.Generator().manual_seed(2)
    k, v, x = (torch.randn((T, h, D), generator=g).to(torch.bfloat16) for h in (Hkv, Hkv, 8))
    outs = []
    for pdl in (False, True):
        q.set_pdl(pdl)
        try:
            t, kd, vd, sd = i32(table), to_cache(kc, "e4m3"), to_cache(vc, "e4m3"), torch.from_numpy(sc.copy()).to(DEV)
            free, count, od_, nd = i32(ids), i32([9]), i32(old), i32(new)
            kk, vv, xx = k.to(DEV), v.to(DEV), x.to(DEV)
            torch.cuda.synchronize()
            _, cu, slots, _, info = q.kv8_block_plan(od_, nd, t, free, count, bs, T)
            q.kv8_append(kk, vv, slots, kd, vd, sd)
            out = q.attn_kv8_paged(xx, kd, vd, sd, t, nd, cu)
            torch.cuda.synchronize()
        finally:
            q.set_pdl(False)
        assert info[3].item() == 0
        outs.append((out.cpu(), bits(kd), bits(vd), sd.cpu(), t.cpu().numpy(), cu.cpu().numpy()))
    assert torch.equal(outs[0][0], outs[1][0]) and np.array_equal(outs[0][1], outs[1][1])
    out, kb, vb, sb, tb, cub = outs[0]
    c = dict(x=torch.cat((x, x[:1])), kc=kb, vc=vb, sc=sb.numpy(), table=tb, ctx=new, cu=cub, masks=None, fmt="e4m3")
    check_attn(torch.cat((out, torch.full_like(out[:1], 7.0))), c)


# --------------------------------------------------------------------------
# attention, many query rows: a wide block table makes the bound of the lengths large, and with it the tcgen05 kernel
# runs (more than 16 rows of up to 128 elements per key/value head)
# --------------------------------------------------------------------------

def widen(c, tokens=1 << 20):
    R, maxb = c["table"].shape
    bs = c["kc"].shape[2]
    wide = np.full((R, tokens // bs), -1, np.int64)
    wide[:, :maxb] = c["table"]
    return dict(c, table=wide)


MANY = [
    # query tokens, context lengths, Hq, Hkv, block, tree
    ([16], [2063], 32, 8, 64, True),
    ([16], [16], 32, 8, 16, True),
    ([12], [128], 32, 8, 16, False),
    ([9], [129], 4, 1, 16, False),
    ([16, 1, 32, 7], [16, 1, 32, 200], 8, 2, 16, True),
    ([11, 0, 16], [1500, 90, 127], 8, 2, 48, False),
    ([40, 33], [40, 300], 4, 2, 32, True),
    ([100], [1000], 4, 1, 128, False),
    ([5, 6, 7], [333, 2500, 64], 48, 4, 32, False),
    ([64], [4000], 3, 3, 256, False),
    ([3], [777], 64, 1, 1024, False),
    ([20] * 9, [(i * 97) % 700 for i in range(9)], 10, 2, 16, False),
]


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("nq,ctx,Hq,Hkv,bs,tree", MANY)
def test_attention_many_rows(q, fmt, nq, ctx, Hq, Hkv, bs, tree):
    rng = np.random.default_rng(sum(ctx) + bs + Hq)
    c = widen(attn_case(rng, nq, ctx, Hq, Hkv, 128, bs, fmt, tree))
    out = run_attn(q, c)
    check_attn(out, c)
    assert torch.equal(run_attn(q, c), out)  # the same bits again


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 112])
def test_attention_many_rows_head_sizes(q, fmt, D):
    rng = np.random.default_rng(D)
    for nq, ctx in (([12], [6000]), ([9, 16, 1], [9, 700, 130])):
        c = widen(attn_case(rng, nq, ctx, 16, 2, D, 48, fmt, True))
        check_attn(run_attn(q, c), c)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_attention_many_rows_masks_and_scales(q, fmt):
    rng = np.random.default_rng(61)
    # rows that see nothing, among ones that do
    c = widen(attn_case(rng, [16, 12], [16, 12], 16, 2, 128, 16, fmt, True))
    c["masks"][:16] = [0, 1, 0, 0xFFFF0000, 0b1111, 0, 0x80000000, 3, 0, 0, 1 << 9, 0, 0, 0, 0, 0x8000]
    out = run_attn(q, c)
    check_attn(out, c)
    assert not out[0].any() and not out[3].any() and not out[15, :, :].isnan().any() and out[1].any()
    # a context shorter than the query tokens
    c = widen(attn_case(rng, [20], [7], 8, 2, 128, 16, fmt, False))
    out = run_attn(q, c)
    check_attn(out, c)
    assert not out[:13].any() and out[13].any()
    # blocks of zero scale, scales that differ by 2^30, large and tiny queries
    c = widen(attn_case(rng, [10, 14], [900, 333], 16, 2, 128, 16, fmt, False))
    c["sc"][::3, :, 1] = 0.0
    c["sc"][1::3, :, 1] *= np.float32(2.0 ** -30)
    c["sc"][::5, :, 0] = 0.0
    c["x"][1] *= 1e-6
    c["x"][2] *= 40.0
    check_attn(run_attn(q, c), c)
    c["sc"][..., 1] = 0.0
    assert not run_attn(q, c)[:24].any()
    c["sc"][..., 1] = np.float32(2.0 ** 40)
    check_attn(run_attn(q, c), c)


def test_attention_many_rows_peaked_bad_blocks_and_lengths(q):
    rng = np.random.default_rng(62)
    c = widen(attn_case(rng, [14], [2600], 16, 4, 128, 32, "i8", False, qstd=30.0))
    check_attn(run_attn(q, c), c)
    check_attn(run_attn(q, c, softmax_scale=1.7), c, 1.7)
    check_attn(run_attn(q, c, softmax_scale=1e-6), c, 1e-6)
    c = widen(attn_case(rng, [10, 12], [700, 190], 16, 2, 128, 16, "i8", False))
    c["table"][0, 3], c["table"][0, 37], c["table"][1, 0] = -1, c["kc"].shape[0], 2 ** 31 - 1
    c["table"][0, 8:16] = -5                             # a whole step of bad blocks
    check_attn(run_attn(q, c), c)
    assert q.device_error(clear=True) == 0x602


def test_attention_many_rows_long(q):
    rng = np.random.default_rng(63)
    check_attn(run_attn(q, c := widen(attn_case(rng, [9], [40001], 4, 1, 128, 64, "e4m3", False))), c)


def test_attention_many_rows_many_requests(q):
    """More requests than leave room for the third ring stage."""
    rng = np.random.default_rng(64)
    c = widen(attn_case(rng, [9] * 1000, [9 + i % 5 for i in range(1000)], 4, 1, 128, 16, "i8", False), 1024)
    check_attn(run_attn(q, c), c)


def test_attention_many_rows_in_a_graph(q):
    rng = np.random.default_rng(65)
    c = widen(attn_case(rng, [16, 10], [900, 40], 8, 2, 128, 16, "i8", False))
    dev = [c["x"].to(DEV), to_cache(c["kc"], "i8"), to_cache(c["vc"], "i8"), torch.from_numpy(c["sc"]).to(DEV),
           i32(c["table"]), i32(c["ctx"]), i32(c["cu"])]
    out = torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16)
    q.attn_kv8_paged(*dev, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_kv8_paged(*dev, out=out)
    for ctx in ([900, 40], [128, 33], [16, 10]):
        dev[5].copy_(i32(ctx))
        for _ in range(2):
            out.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        check_attn(out.cpu(), dict(c, ctx=np.array(ctx)))


# --------------------------------------------------------------------------
# norm
# --------------------------------------------------------------------------

TD = {"f32": torch.float32, "bf16": torch.bfloat16}


def norm_inputs(M, K, xd, rd, wd, seed):
    x = synth.normal_f32((M, K), 1.0, seed, 0).to(TD[xd])
    r = None if rd is None else (synth.normal_f32((M, K), 3.0, seed, 1)).to(TD[rd])
    if r is not None:
        r[:, ::61] *= 20
    w = (1 + synth.normal_f32((K,), 0.3, seed, 2)).to(TD[wd])
    h = x.float() if r is None else (x.float() + r.float()).to(TD[rd]).float()
    return x, r, w, h


NORM = [(1, 32, "f32", "f32", "bf16"), (1, 4096, "f32", "f32", "bf16"), (3, 4096, "bf16", "bf16", "f32"),
        (16, 7168, "bf16", "f32", "bf16"), (5, 12288, "f32", "bf16", "bf16"), (2, 32768, "f32", "f32", "f32"),
        (33, 96, "bf16", "bf16", "bf16"), (2, 8224, "bf16", None, "bf16"), (4, 16416, "f32", "f32", "bf16"),
        (700, 2080, "f32", "bf16", "bf16")]


@pytest.mark.parametrize("M,K,xd,rd,wd", NORM)
def test_norm_bf16(q, M, K, xd, rd, wd):
    x, r, w, h = norm_inputs(M, K, xd, rd, wd, 31)
    y, ho = q.rmsnorm_residual(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=1e-5)
    torch.cuda.synchronize()
    if r is None:
        assert ho is None
    else:
        assert torch.equal(ho.float().cpu(), h)
    ref, _ = od.rmsnorm(h.double().numpy(), w.double().numpy(), 1e-5)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref))


@pytest.mark.parametrize("had", [False, True])
@pytest.mark.parametrize("M,K,xd,rd,wd", NORM)
def test_norm_i8(q, M, K, xd, rd, wd, had):
    x, r, w, h = norm_inputs(M, K, xd, rd, wd, 37)
    if M > 2:
        x[1] = 0
        h[1] = 0
        if r is not None:
            r[1] = 0
    sb = synth.sign_bits(K, 38, 0) if had else None
    qd, sd, ho = q.rmsnorm_residual_i8(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=1e-5,
                                       sign_bits=None if sb is None else sb.to(DEV))
    torch.cuda.synchronize()
    if r is not None:
        assert torch.equal(ho.float().cpu(), h)
    z, mag = od.rmsnorm(h.double().numpy(), w.double().numpy(), 1e-5, None if sb is None else sb.numpy())
    err = 48 * 2.0 ** -24 * mag
    amax, emax = np.abs(z).max(-1), err.max(-1)
    s = sd.double().cpu().numpy()
    assert np.all(np.abs(s - amax / 127) <= emax / 127 + 2.0 ** -23 * amax / 127)
    codes = qd.double().cpu().numpy()
    assert np.abs(codes).max() <= 127
    live = s > 0
    assert np.array_equal(live, amax > 0) and not codes[~live].any()
    step = s[live, None]
    off = np.abs(codes[live] * step - z[live])
    assert np.all(off <= step * 0.5 + err[live] + 127 * 2.0 ** -23 * step)


def test_norm_in_place_and_transform_agree_with_the_quantizer(q):
    M, K = 16, 4096
    x, r, w, h = norm_inputs(M, K, "f32", "f32", "bf16", 41)
    sb = synth.sign_bits(K, 41, 5).to(DEV)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    y, ho = q.rmsnorm_residual(xd, wd, residual=rd.clone())
    res = rd.clone()
    y2, same = q.rmsnorm_residual(xd, wd, residual=res, residual_out=res)
    assert same is res and torch.equal(y, y2) and torch.equal(res, ho)
    # a weight that makes y a bf16 number: the codes are the quantizer's own, bit for bit
    yb, _ = q.rmsnorm_residual(xd, wd, residual=rd)
    one = torch.ones(K, device=DEV)
    xs = (torch.randint(-7, 8, (M, K), generator=torch.Generator().manual_seed(3)).float() * 8).to(DEV)
    xs[:, 0] = 8
    unit = xs / xs.square().mean(-1, keepdim=True).sqrt()
    q8, s8, _ = q.rmsnorm_residual_i8(unit, one, sign_bits=sb, eps=0.0)
    qr, sr = q.hadamard32_quant_i8(xs.to(torch.bfloat16), sb)
    torch.cuda.synchronize()
    assert (q8.int() - qr.int()).abs().max().item() <= 1  # the rows differ by a factor, rounded once
    assert yb.dtype == torch.bfloat16


def test_norm_feeds_the_int8_product(q):
    """norm -> codes -> exact int8 product against the float64 product of the codes."""
    M, K, N = 8, 1024, 192
    x, r, w, h = norm_inputs(M, K, "f32", "f32", "bf16", 43)
    sb = synth.sign_bits(K, 43, 5)
    qa, sa, _ = q.rmsnorm_residual_i8(x.to(DEV), w.to(DEV), residual=r.to(DEV), sign_bits=sb.to(DEV))
    w8 = torch.randint(-127, 128, (N, K), generator=torch.Generator().manual_seed(4), dtype=torch.int8)
    c = q.gemm_w8a8_i32(qa, w8.to(DEV))
    torch.cuda.synchronize()
    assert np.array_equal(c.cpu().numpy(), (qa.cpu().double() @ w8.double().T).to(torch.int32).numpy())


def test_python_refusals(q):
    z = torch.zeros
    kc = z((2, 2, 16, 64), device=DEV, dtype=torch.int8)
    sc = z((2, 2, 2), device=DEV)
    x = z((1, 2, 64), device=DEV, dtype=torch.bfloat16)
    one = i32([1])
    tab = i32([[0, 1]])
    cu = i32([0, 1])
    with pytest.raises(ValueError):
        q.attn_kv8_paged(x, kc, kc.view(torch.float8_e4m3fn), sc, tab, one, cu)
    with pytest.raises(ValueError):
        q.attn_kv8_paged(x.float(), kc, kc, sc, tab, one, cu)
    with pytest.raises(ValueError):
        q.attn_kv8_paged(x, kc, kc, sc, tab.long(), one, cu)
    with pytest.raises(ValueError):
        q.attn_kv8_paged(x, kc, kc, sc[:1], tab, one, cu)
    with pytest.raises(ValueError):
        q.attn_kv8_paged(x, kc, kc, sc, tab, one, i32([0, 1, 1]))
    with pytest.raises(q.QGError):
        q.attn_kv8_paged(z((1, 3, 64), device=DEV, dtype=torch.bfloat16), kc, kc, sc, tab, one, cu)
    with pytest.raises(ValueError):
        q.kv8_append(x, x[:, :1], one, kc, kc, sc)
    with pytest.raises(ValueError):
        q.kv8_append(x.half(), x.half(), one, kc, kc, sc)
    with pytest.raises(ValueError):
        q.kv8_append(x.transpose(1, 2), x.transpose(1, 2), one, kc, kc, sc)
    with pytest.raises(ValueError):
        q.kv8_read(torch.zeros(1, device=DEV, dtype=torch.int64), kc, kc, sc)
    with pytest.raises(ValueError):
        q.kv8_block_plan(one, i32([1, 2]), tab, one, one, 16, 4)
    with pytest.raises(q.QGError):
        q.rmsnorm_residual(z((1, 33), device=DEV), z(33, device=DEV))
    with pytest.raises(ValueError):
        q.rmsnorm_residual(z((1, 64), device=DEV), z(32, device=DEV))
    with pytest.raises(ValueError):
        q.rmsnorm_residual(z((1, 64), device=DEV, dtype=torch.float16), z(64, device=DEV))


# --------------------------------------------------------------------------
# guard bands
# --------------------------------------------------------------------------

BAND = 4096


def banded(shape, dtype):
    """A tensor between two bands of a fixed byte pattern, and the whole buffer."""
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((2 * BAND + n + 64,), 0xA5, device=DEV, dtype=torch.uint8)
    return buf[BAND:BAND + n].view(dtype).view(shape), (buf, n)


def intact(band):
    buf, n = band
    return bool((buf[:BAND] == 0xA5).all()) and bool((buf[BAND + n:] == 0xA5).all())


def test_writes_stay_inside(q):
    rng = np.random.default_rng(51)
    bands = []

    def make(shape, dtype):
        t, b = banded(shape, dtype)
        bands.append(b)
        return t
    # plan
    old, new, table, free, count = plan_state(rng, 37, 16, 90, 30, 1)
    tokens = int(np.maximum(new - old, 0).sum())
    t = make(table.shape, torch.int32).copy_(i32(table))
    f = make(free.shape, torch.int32).copy_(i32(free))
    out = dict(free_count_out=make((1,), torch.int32), cu_new=make((38,), torch.int32),
               slot_map=make((tokens + 1,), torch.int32), positions=make((tokens + 1,), torch.int32),
               info=make((4,), torch.int32), workspace=make((16,), torch.uint8).zero_())
    q.kv8_block_plan(i32(old), i32(new), t, f, i32([count]), 16, tokens + 1, **out)
    # append and attention
    for D, bs, fmt in ((128, 16, "i8"), (64, 48, "e4m3"), (256, 32, "i8"), (48, 16, "e4m3")):
        H, nb = 3, 4
        kc, vc, sc = random_cache(rng, nb, H, bs, D, fmt)
        kd = make(kc.shape, DT[fmt])
        vd = make(vc.shape, DT[fmt])
        kd.view(torch.uint8).copy_(torch.from_numpy(kc))
        vd.view(torch.uint8).copy_(torch.from_numpy(vc))
        sd = make(sc.shape, torch.float32).copy_(torch.from_numpy(sc))
        slots = list(range(bs - 3, bs)) + list(range((nb - 1) * bs, nb * bs))
        k = torch.randn((len(slots), H, D), device=DEV)
        q.kv8_append(k, k, i32(slots), kd, vd, sd)
        x = torch.randn((5, 9, D), device=DEV).to(torch.bfloat16)
        need = q.lib().qg_attn_kv8_workspace_size(9, H, D)
        ws = make((max(16, need),), torch.uint8).zero_()
        o = make((5, 9, D), torch.bfloat16)
        q.attn_kv8_paged(x, kd, vd, sd, i32([[3, 0, 1, 2], [1, 2, 0, 3]]), i32([4 * bs, bs + 1]), i32([0, 3, 5]), out=o,
                         workspace=ws)
        torch.cuda.synchronize()
        assert torch.isfinite(o).all()
    # attention with many rows
    kc, vc, sc = random_cache(rng, 9, 2, 16, 128, "i8")
    x = torch.randn((24, 16, 128), device=DEV).to(torch.bfloat16)
    table = np.full((2, 65536), -1)
    table[0, :9], table[1, :9] = np.arange(9), np.arange(9)[::-1]
    need = q.lib().qg_attn_kv8_workspace_size(16, 2, 128)
    o = make((24, 16, 128), torch.bfloat16)
    q.attn_kv8_paged(x, to_cache(kc, "i8"), to_cache(vc, "i8"), torch.from_numpy(sc).to(DEV), i32(table), i32([144, 130]),
                     i32([0, 10, 24]), out=o, workspace=make((need,), torch.uint8).zero_())
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    # norm
    for M, K in ((3, 96), (2, 8224)):
        x = torch.randn((M, K), device=DEV)
        w = torch.ones(K, device=DEV)
        ro = make((M, K), torch.float32)
        q.rmsnorm_residual(x, w, residual=x, residual_out=ro, out=make((M, K), torch.bfloat16))
        q.rmsnorm_residual_i8(x, w, residual=x, residual_out=ro, q=make((M, K), torch.int8),
                              scale=make((M,), torch.float32))
    torch.cuda.synchronize()
    assert all(intact(b) for b in bands)


@pytest.mark.parametrize("D", [16, 64, 96, 128, 256])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_pieces_stay_in_the_queried_workspace(q, D, wide):
    """Contexts split over all CTAs (every CTA has a piece of two items) with a workspace of exactly the queried size,
    16 MB of a fixed pattern behind it; with a wide table heads of up to 128 run on the tcgen05 kernel."""
    rng = np.random.default_rng(71 + D)
    Hq, Hkv = 20, 4
    c = attn_case(rng, [9, 12, 5], [9000, 4100, 6007], Hq, Hkv, D, 64, "i8", False)
    if wide:
        c = widen(c)
    need, behind = q.lib().qg_attn_kv8_workspace_size(Hq, Hkv, D), 16 << 20
    buf = torch.full((BAND + need + behind,), 0xA5, device=DEV, dtype=torch.uint8)
    ws = buf[BAND:BAND + need].zero_()
    for _ in range(2):
        check_attn(run_attn(q, c, workspace=ws), c)
        assert intact((buf, need))


# --------------------------------------------------------------------------
# workspaces and stream captures
# --------------------------------------------------------------------------

def on_device(c):
    return [c["x"].to(DEV), to_cache(c["kc"], c["fmt"]), to_cache(c["vc"], c["fmt"]), torch.from_numpy(c["sc"]).to(DEV),
            i32(c["table"]), i32(c["ctx"]), i32(c["cu"])]


def captured(st, calls):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        calls()
    return g


def test_a_capture_has_a_workspace_of_its_own(q):
    """Also where the captured stream has had an eager call: the graph's own memory holds the workspace."""
    rng = np.random.default_rng(81)
    c = attn_case(rng, [1, 2], [3000, 400], 8, 2, 128, 16, "i8", False)
    dev, out = on_device(c), torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q.attn_kv8_paged(*dev, out=out)                  # a workspace is kept for the stream
    st.synchronize()
    g = captured(st, lambda: (q.attn_kv8_paged(*dev, out=out), q.attn_kv8_paged(*dev, out=out)))
    need = q.lib().qg_attn_kv8_workspace_size(8, 2, 128)
    own = sum(s["total_size"] for s in torch.cuda.memory_snapshot() if tuple(s["segment_pool_id"]) == tuple(g.pool()))
    assert own >= need
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_attn(out.cpu(), c)


def test_a_graph_outlives_the_kept_workspace(q):
    """An eager call that needs a larger workspace on the captured stream replaces the kept one; what then gets its
    memory is not written by replays."""
    rng = np.random.default_rng(82)
    small = attn_case(rng, [2, 1], [5000, 700], 8, 2, 256, 32, "i8", False)
    large = attn_case(rng, [1, 1], [4000, 60], 8, 2, 128, 32, "i8", False)
    st = torch.cuda.Stream()
    ds, dl = on_device(small), on_device(large)
    outs = [torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16) for c in (small, large)]
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        q.attn_kv8_paged(*ds, out=outs[0])
    g = captured(st, lambda: q.attn_kv8_paged(*ds, out=outs[0]))
    with torch.cuda.stream(st):
        q.attn_kv8_paged(*dl, out=outs[1])
        fill = [torch.full((4 << 20,), 0x5A, device=DEV, dtype=torch.uint8) for _ in range(8)]
        outs[0].fill_(7.0)
        for _ in range(3):
            g.replay()
            q.attn_kv8_paged(*dl, out=outs[1])
    st.synchronize()
    assert all(bool((f == 0x5A).all()) for f in fill)
    check_attn(outs[0].cpu(), small)
    check_attn(outs[1].cpu(), large)


@pytest.mark.parametrize("wide", [False, True])
def test_graphs_of_one_stream_replayed_side_by_side(q, wide):
    """Two graphs captured on a stream that has had eager calls, replayed on two streams next to further eager ones."""
    rng = np.random.default_rng(83)
    cases = [attn_case(rng, [9, 2], [6000, 500], 16, 2, 128, 16, "i8", False) for _ in range(3)]
    if wide:
        cases = [widen(c) for c in cases]
    dev = [on_device(c) for c in cases]
    outs = [torch.full(c["x"].shape, 7.0, device=DEV, dtype=torch.bfloat16) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    with torch.cuda.stream(streams[0]):
        q.attn_kv8_paged(*dev[0], out=outs[0])
    graphs = [captured(streams[0], lambda i=i: q.attn_kv8_paged(*dev[i], out=outs[i])) for i in (1, 2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                if i == 0:
                    q.attn_kv8_paged(*dev[0], out=outs[0])
                else:
                    graphs[i - 1].replay()
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        check_attn(out.cpu(), c)


def test_plans_captured_on_one_stream_replayed_side_by_side(q):
    """The plan's ticket too: several CTAs a call, the count written by the last."""
    rng = np.random.default_rng(84)
    streams = [torch.cuda.Stream() for _ in range(3)]
    states = [plan_state(rng, 300, 16, 90, 60, 5) for _ in range(3)]
    tokens = [int(np.maximum(n - o, 0).sum()) for o, n, *_ in states]
    args = [[i32(o), i32(n), i32(t), i32(f), i32([c])] for o, n, t, f, c in states]
    outs = [dict(free_count_out=i32([-9]), cu_new=i32([0] * 301), slot_map=i32([0] * t), positions=i32([0] * t),
                 info=i32([9] * 4)) for t in tokens]
    calls = [lambda i=i: q.kv8_block_plan(*args[i], 16, tokens[i], **outs[i]) for i in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        calls[0]()
    graphs = [captured(streams[0], c) for c in calls[1:]]
    torch.cuda.synchronize()
    want = [od.block_plan(o, n, t, f, c, 16, k) for (o, n, t, f, c), k in zip(states, tokens)]
    for _ in range(10):
        for i, (o, n, t, f, c) in enumerate(states):     # as they were
            args[i][2].copy_(i32(t)), args[i][3].copy_(i32(f)), outs[i]["free_count_out"].fill_(-9)
        torch.cuda.synchronize()
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                calls[0]() if i == 0 else graphs[i - 1].replay()
        torch.cuda.synchronize()
        for i in range(3):
            got = [args[i][2], args[i][3]] + [outs[i][k] for k in ("free_count_out", "cu_new", "slot_map", "positions",
                                                                     "info")]
            for g, w in zip(got, want[i]):
                assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


def test_captured_products_have_workspaces_of_their_own(q):
    """The skinny product and the fused int8 product likewise, and a workspace first made for a given stream is zeroed
    there."""
    w4 = synth.w4_weights(512, 1024, seed=5, slot=0, device=DEV)
    x = synth.bf16_normal((16, 1024), seed=5, slot=1, device=DEV)
    sb = synth.sign_bits(1024, 5, 2).to(DEV)
    w8, s8 = q.hadamard32_quant_i8(synth.bf16_normal((256, 1024), seed=5, slot=3, device=DEV), sb)
    assert q.lib().qg_skinny_workspace_size(16, 512, 1024, 64) + q.lib().qg_w8a8_hadamard_workspace_size(16, 1024) > 0
    want = q.qgemm_w4a16_skinny(*w4, x), q.gemm_w8a8_hadamard(x, sb, w8, s8)
    outs = [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    kept = [q.skinny_workspace(1, DEV, st), q._workspace("w8a8", 1 << 16, DEV, st)]

    def calls():
        q.qgemm_w4a16_skinny(*w4, x, y=outs[0], stream=st)
        q.gemm_w8a8_hadamard(x, sb, w8, s8, y=outs[1], stream=st)

    calls()
    st.synchronize()
    inside = []
    g = captured(st, lambda: (inside.extend((q.skinny_workspace(1, DEV), q._workspace("w8a8", 1 << 16, DEV, None))), calls()))
    assert q.skinny_workspace(1, DEV, st).data_ptr() == kept[0].data_ptr()
    pool = [s for s in torch.cuda.memory_snapshot() if tuple(s["segment_pool_id"]) == tuple(g.pool())]
    for ws in inside:
        assert any(s["address"] <= ws.data_ptr() < s["address"] + s["total_size"] for s in pool)
    for _ in range(2):
        for o in outs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# --------------------------------------------------------------------------
# attention: scores
# --------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 10])
def test_attention_scores_of_small_codes(q, D, fmt, G):
    """Keys of codes +-1 under positive queries: the score's error goes by sum |q k|, not by the queries' sum. Both
    tokens of a context have the same score (the query's halves are equal, the second key has its halves exchanged) and
    opposite values, so what the result differs from 0 by is the scores' error."""
    rng = np.random.default_rng(91 + D)
    R, Hkv, bs = 64, 8, 16
    c = attn_case(rng, [1] * R, [2] * R, G * Hkv, Hkv, D, bs, fmt, False)
    one = {"i8": (1, 255), "e4m3": (0x38, 0xB8)}[fmt]
    for r in range(R):
        b = c["table"][r, 0]
        k = np.where(rng.random((Hkv, D)) < 0.5, *one).astype(np.uint8)
        c["kc"][b, :, 0], c["kc"][b, :, 1] = k, np.roll(k, D // 2, -1)
        c["vc"][b, :, 0] = {"i8": 100, "e4m3": 0x6C}[fmt]
        c["vc"][b, :, 1] = {"i8": 256 - 100, "e4m3": 0xEC}[fmt]
    half = np.exp(rng.standard_normal(tuple(c["x"].shape[:2]) + (D // 2,)))
    c["x"] = torch.from_numpy(np.concatenate((half, half), -1)).to(torch.bfloat16)
    c["sc"][..., 0] = 1.0
    scale = 0.01 / ((D + 8) * 2.0 ** -23 * float(c["x"].double().sum(-1).max()))
    check_attn(run_attn(q, c, softmax_scale=scale), c, scale)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_rows_do_not_touch_one_another(q, wide, tree):
    """Infinite and NaN query elements stay in their own rows, and rows of very different sizes keep their precision,
    also where many rows share a pass over the cache."""
    rng = np.random.default_rng(95)
    c = attn_case(rng, [14, 9], [1500, 333], 16, 4, 128, 32, "i8", tree, qstd=1.5)
    if wide:
        c = widen(c)
    for (t, h), f in {(1, 2): 2.0 ** 30, (3, 5): 2.0 ** -17, (4, 5): 2.0 ** 17, (6, 9): 2.0 ** 100, (7, 9): 0.0,
                      (16, 15): 2.0 ** 20, (17, 3): 2.0 ** -100}.items():
        c["x"][t, h] = (c["x"][t, h].float() * f).to(torch.bfloat16)
    check_attn(run_attn(q, c), c)
    bad = [(0, 1), (2, 5), (5, 6), (18, 0), (22, 15)]
    clean = dict(c, x=c["x"].clone())
    for i, (t, h) in enumerate(bad):
        clean["x"][t, h] = 0.0
        c["x"][t, h, 7 * i] = (math.inf, math.nan, -math.inf)[i % 3]
    out = run_attn(q, c)
    for t, h in bad:
        assert bool(out[t, h].isnan().any())
        out[t, h] = run_attn(q, clean)[t, h]
    check_attn(out, clean)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,ctx,wide", [(1, 1, False), (1, 3000, False), (16, 16, True), (16, 3000, True)])
def test_attention_scores_far_below_zero(q, D, nq, ctx, wide):
    """Every seen score is some -1e31: values that are all alike come out, whatever the weights."""
    c = attn_case(np.random.default_rng(97), [nq], [ctx], 8, 2, D, 16, "i8", False)
    if wide:
        c = widen(c)
    c["x"][:] = -1e30
    c["kc"][:], c["vc"][:], c["sc"][:] = 1, 100, 1.0
    out = run_attn(q, c)[:nq].float()
    assert bool(((out - 100.0).abs() <= 100 * 2.0 ** -8).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_scores_past_the_steps_of_fp32(q, D):
    """Scores of 2^27, where fp32 has steps of 16: a later token one step above the largest so far takes all weight."""
    rng = np.random.default_rng(98)
    apart = 128 if D == 256 else 256                      # tokens of a step: one warp takes these, one after the other
    c = attn_case(rng, [1], [2 * apart + 80], 8, 2, D, 16, "i8", False)
    c["kc"][:] = 0
    c["sc"][:] = 1.0
    c["x"][:] = 0.0
    c["x"][..., 0], c["x"][..., 1] = 2.0 ** 27, 16.0
    scale = float(np.float32(np.log(2.0)))               # the scores are q . k in units of log 2
    assert np.float32(scale) * np.float32(np.log2(np.e)) == 1
    for j in (1, 2, 3):
        tok = 3 + (j - 1) * apart
        b = c["table"][0, tok // 16]
        c["kc"][b, :, tok % 16, 0], c["kc"][b, :, tok % 16, 1] = 1, j
    want = torch.from_numpy(c["vc"][b, :, tok % 16].view(np.int8).astype(np.float32)).repeat_interleave(4, 0)
    out = run_attn(q, c, softmax_scale=scale)[0].float()
    assert bool(((out - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -16 * 256).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cu", [[0, 12, 9, 20], [0, 12, 16, 24], [-1, 12, 16, 20], [3, 2, 1, 0]])
def test_attention_query_bounds_that_do_not_ascend(q, cu, wide):
    """Reported, and nothing is written."""
    c = attn_case(np.random.default_rng(99), [8, 8, 4], [300, 40, 20], 8, 2, 128, 16, "i8", False)
    c["x"] = c["x"][:20]
    if wide:
        c = widen(c)
    c["cu"] = np.array(cu)
    assert bool((run_attn(q, c) == 7.0).all())
    assert q.device_error(clear=True) == 0x604
    c["cu"] = np.array([0, 8, 8, 20])
    check_attn(run_attn(q, c), c)


# --------------------------------------------------------------------------
# norm of many rows: several steps a thread, and rows of more than 8192 elements
# --------------------------------------------------------------------------

NORM_MANY = [(700, 7168, "bf16", "bf16", "bf16"), (611, 8192, "f32", "f32", "f32"), (640, 4128, "f32", "bf16", "bf16"),
             (609, 4096, "bf16", "f32", "f32"), (615, 5152, "bf16", None, "bf16"), (612, 12288, "f32", "f32", "bf16")]


@pytest.mark.parametrize("M,K,xd,rd,wd", NORM_MANY)
def test_norm_bf16_of_many_rows(q, M, K, xd, rd, wd):
    test_norm_bf16(q, M, K, xd, rd, wd)


@pytest.mark.parametrize("had", [False, True])
@pytest.mark.parametrize("M,K,xd,rd,wd", NORM_MANY)
def test_norm_i8_of_many_rows(q, M, K, xd, rd, wd, had):
    test_norm_i8(q, M, K, xd, rd, wd, had)
