"""The decode-layer example: every stage of its steps against the oracle, given
the stage's own inputs (prompts, single tokens, a draft tree, a rollback)."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import decode as od

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    from skinny_gemm_qgemv_gb300 import build
    build.build()
    import decode_layer
    import skinny_gemm_qgemv_gb300 as q
    q.device_error(clear=True)
    yield decode_layer
    assert q.device_error(clear=True) == 0


def w4(w, x):
    y, ad = oracle.w4a16(*(t.cpu() for t in w), x.cpu())
    return y, oracle.tolerance(ad)


def check_step(layer, t, before, cache, new_lens, bs, tree):
    table, free, count, k0, v0, s0, lens0 = before
    M = t["x"].shape[0]
    # norm and projections
    h = (t["x"] + t["old_residual"]).cpu()
    assert torch.equal(t["residual1"].cpu(), h)
    ref, _ = od.rmsnorm(h.double().numpy(), layer.norm1.double().cpu().numpy(), 1e-6)
    assert np.all(np.abs(t["h1"].double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref))
    # plan
    want = od.block_plan(lens0, new_lens, table, free, count, bs, M)
    got = (cache.table, cache.free, cache.count, t["cu"], t["slots"], t["positions"], t["info"])
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    # append
    kb, s_k = od.append(t["k"].cpu().numpy(), t["slots"].cpu().numpy(), k0, s0[..., 0], od.I8, len(k0), bs)
    vb, s_v = od.append(t["v"].cpu().numpy(), t["slots"].cpu().numpy(), v0, s0[..., 1], od.I8, len(k0), bs)
    assert np.array_equal(cache.k.view(torch.uint8).cpu().numpy(), kb)
    assert np.array_equal(cache.v.view(torch.uint8).cpu().numpy(), vb)
    scales = np.stack((s_k, s_v), -1)
    assert np.array_equal(cache.scales.cpu().numpy(), scales)
    # attention (the bound of test_gpu_decode_ops.py)
    D = layer.head_dim
    ref, mag, qk, n, vmax = od.attention(t["q"].float().cpu().numpy(), kb, vb, scales, cache.table.cpu().numpy(), new_lens,
                                         t["cu"].cpu().numpy(), od.I8, D ** -0.5, tree)
    qk, n, vmax = qk[:, :, None], n[:, :, None], vmax[:, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * qk + n * 2.0 ** -24) * mag + \
        n * 2.0 ** -25 * vmax
    assert np.all(np.abs(t["attn"].double().cpu().numpy() - ref) <= tol)
    # output projection, second norm, down projection
    y, tol = w4(layer.wo, t["attn"].flatten(1))
    assert np.all(np.abs(t["o"].double().cpu().numpy() - y) <= tol)
    h2 = (t["o"] + t["residual1"]).double().cpu().numpy()
    z, mag = od.rmsnorm(h2, layer.norm2.double().cpu().numpy(), 1e-6, layer.sign_bits.cpu().numpy())
    step = t["s"].double().cpu().numpy()[:, None]
    off = np.abs(t["h8"].double().cpu().numpy() * step - z)
    assert np.all(off <= step * 0.5 + 48 * 2.0 ** -24 * mag + 127 * 2.0 ** -23 * step)
    y, tol = w4(layer.wdown, t["act"])
    assert np.all(np.abs(t["y"].double().cpu().numpy() - y) <= tol)


def test_decode_layer_steps(ex):
    torch.manual_seed(3)
    R, hidden = 3, 512
    layer = ex.DecodeLayer(hidden, heads=4, kv_heads=2, head_dim=64, intermediate=512, seed=2)
    cache = ex.PagedCache(R, num_blocks=40, max_blocks=12, Hkv=2, D=64)
    cache.k.fill_(5)                                      # stale codes: a new block starts from zeros
    lens = [0] * R

    def step(new, tree=None):
        nonlocal lens
        M = sum(b - a for a, b in zip(lens, new))
        before = (cache.table.cpu().numpy(), cache.free.cpu().numpy(), cache.count.item(),
                  cache.k.view(torch.uint8).cpu().numpy(), cache.v.view(torch.uint8).cpu().numpy(),
                  cache.scales.cpu().numpy(), list(lens))
        x, res = torch.randn(M, hidden, device="cuda"), torch.randn(M, hidden, device="cuda") * 2
        words = None if tree is None else ex.tree_words(tree).repeat(R)
        _, t = layer.step(x, res, cache, torch.tensor(new, dtype=torch.int32, device="cuda"), tree=words)
        torch.cuda.synchronize()
        check_step(layer, t, before, cache, new, 16, None if words is None else words.cpu().numpy().view(np.uint32))
        lens = list(new)

    step([3, 15, 14])
    step([4, 16, 15])
    step([5, 17, 16])
    step([10, 22, 21], tree=[-1, 0, 0, 2, 1])
    cache.resize(torch.tensor([6, 17, 16], dtype=torch.int32, device="cuda"), 1)   # most drafts rejected
    lens = [6, 17, 16]
    step([7, 18, 17])


def test_example_runs(ex, capsys):
    ex.main()
    assert "free blocks" in capsys.readouterr().out


def test_a_refused_plan_leaves_the_cache_as_it_was(ex):
    """More tokens than the pool has blocks for: lengths, table and stack stay, and the next steps are sound."""
    layer = ex.DecodeLayer(512, heads=4, kv_heads=2, head_dim=64, intermediate=512, seed=4)
    cache = ex.PagedCache(2, num_blocks=3, max_blocks=8, Hkv=2, D=64)
    lens = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(*new):
        M = max(1, sum(new) - int(cache.lens.sum()))
        return layer.step(torch.randn(M, 512, device="cuda"), torch.randn(M, 512, device="cuda"), cache, lens(*new))

    _, t = step(14, 10)
    assert t["info"].tolist() == [24, 2, 0, 0] and cache.lens.tolist() == [14, 10]
    before = cache.table.clone(), cache.free.clone(), cache.count.clone(), cache.k.clone(), cache.scales.clone()
    _, t = step(20, 20)
    assert t["info"].tolist() == [0, 0, 0, 1] and cache.lens.tolist() == [14, 10]
    for a, b in zip(before, (cache.table, cache.free, cache.count, cache.k, cache.scales)):
        assert torch.equal(a, b)
    y, t = step(17, 11)
    assert t["info"].tolist() == [4, 1, 0, 0] and bool(torch.isfinite(y).all())
    *_, info = cache.resize(lens(0, 0), 1)
    assert info.tolist() == [0, 0, 3, 0]
    assert cache.count.item() == 3 and sorted(cache.free.tolist()) == [0, 1, 2]
