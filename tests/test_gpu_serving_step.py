"""The serving step's operators together, as the decode-layer example uses them:
norms and rotation, append, attention with a shared prefix, the output head and
the sampler, each against the oracle given its own inputs, eager and captured."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import decode as od
from test_gpu_serving_ops import check_row, rope_ref

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


def i32(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,drafts", [(64, 1), (128, 1), (64, 4), (256, 2)])
def test_serving_steps(ex, D, drafts):
    torch.manual_seed(D)
    hidden, requests = 512, 5
    layer = ex.DecodeLayer(hidden, heads=4, kv_heads=2, head_dim=D, intermediate=512, seed=1)
    head = ex.Head(hidden, vocabulary=3001, seed=1)
    cache = ex.PagedCache(requests, num_blocks=60, max_blocks=12, Hkv=2, D=D)
    rows = lambda m: (torch.randn(m, hidden, device="cuda"), torch.randn(m, hidden, device="cuda"))  # noqa: E731
    # two prefixes (requests 0 and 1); requests 2 and 3 begin with the first, 4 with the second
    layer.step(*rows(21), cache, i32(21, 0, 0, 0, 0))
    layer.step(*rows(9), cache, i32(21, 9, 0, 0, 0))
    cu_req, offset = i32(2, 4, 5), i32(0, 0, 21, 21, 9)
    words = ex.tree_words([-1, 0, 0, 1][:drafts]).repeat(3) if drafts > 1 else None
    for step in range(1, 4):
        n, M = step * drafts, 3 * drafts
        x, residual = rows(M)
        y, t = layer.step(x, residual, cache, i32(21, 9, n, n, n), tree=words, shared=(cu_req, offset))
        torch.cuda.synchronize()
        assert t["info"].tolist()[3] == 0
        # positions count the prefix
        assert t["positions"].tolist() == [o + n - drafts + i for o in (21, 21, 9) for i in range(drafts)]
        pos, freq = t["positions"].cpu()[None], layer.inv_freq.cpu()
        for raw, w, got in ((t["raw_q"], layer.qnorm, t["q"]), (t["raw_k"], layer.knorm, t["k"])):
            ref, mag, turn = rope_ref(raw.cpu(), w.cpu(), 1e-6, pos, freq, np.zeros(len(freq), int), True)
            tol = (2.0 ** -19 + turn * 2.0 ** -51) * mag + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
        table, lens = cache.table.cpu().numpy(), cache.lens.tolist()
        kb, vb = (c.view(torch.uint8).cpu().numpy() for c in (cache.k, cache.v))
        ref, mag, qk, seen, vmax = od.attention_shared(
            t["q"].float().cpu().numpy(), kb, vb, cache.scales.cpu().numpy(), table[:2], lens[:2], [2, 4, 5], table, lens,
            t["cu"].cpu().numpy(), od.I8, D ** -0.5, None if words is None else words.cpu().numpy().view(np.uint32))
        qk, seen, vmax = qk[..., None], seen[..., None], vmax[..., None]
        assert seen.min() > 9 and 21 < seen.max() <= 21 + n
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * qk + seen * 2.0 ** -24 + 2.0 ** -20) * mag + \
            seen * 2.0 ** -25 * vmax
        assert np.all(np.abs(t["attn"].double().cpu().numpy() - ref) <= tol)
        # the head and the draw
        u = torch.rand(M, device="cuda")
        temp = torch.tensor([0.0, 0.7, 1.3] * drafts, device="cuda")
        tokens, probs, logits = head.step(y, residual, u, temperature=temp, top_k=i32(*[40] * M),
                                          top_p=torch.full((M,), 0.9, device="cuda"))
        h = (y + residual).double().cpu().numpy()
        z, _ = od.rmsnorm(h, head.norm.double().cpu().numpy(), 1e-6)
        want, size = oracle.w4a16(*(w.cpu() for w in head.w), torch.from_numpy(z).to(torch.bfloat16))
        # (a row's bf16 rounding of the norm may differ by one unit where it is near a tie)
        off = np.abs(logits.double().cpu().numpy() - want)
        assert np.all(off <= oracle.tolerance(size) + 2.0 ** -7 * size)
        for m in range(M):
            check_row(logits[m].cpu().numpy(), float(u[m]), int(tokens[m]), float(probs[m]), float(temp[m]), 40,
                      np.float32(0.9), 0.0)


def test_serving_step_captured(ex):
    """The step's operators in one graph, replayed with other inputs, against the same calls made eagerly."""
    import skinny_gemm_qgemv_gb300 as lib
    torch.manual_seed(9)
    T, Hq, Hkv, D, bs, V = 6, 8, 2, 128, 16, 20000
    nb = 120
    kc, vc = (torch.zeros((nb, Hkv, bs, D), dtype=torch.int8, device="cuda") for _ in range(2))
    sc = torch.zeros((nb, Hkv, 2), device="cuda")
    pre = torch.arange(50, dtype=torch.int32, device="cuda")[None].contiguous()
    lib.kv8_append(torch.randn(790, Hkv, D, device="cuda"), torch.randn(790, Hkv, D, device="cuda"),
                   torch.arange(790, dtype=torch.int32, device="cuda"), kc, vc, sc)
    table = torch.arange(50, 50 + T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens, cu, slots = i32(*[1] * T), torch.arange(T + 1, dtype=torch.int32, device="cuda"), \
        (torch.arange(T, dtype=torch.int32, device="cuda") + 50) * bs
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    w, pos, u = torch.ones(D, device="cuda"), i32(*[790] * T), torch.rand(T, device="cuda")
    head = torch.randn(Hq * D, V, device="cuda") * 0.2
    fused = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda")
    temp = torch.full((T,), 0.9, device="cuda")

    def step(fused, u):
        q, k, v = (fused[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        q, k = lib.qk_norm_rope(q, k, pos, freq, q_weight=w, k_weight=w)
        lib.kv8_append(k, v, slots, kc, vc, sc)
        o = lib.attn_kv8_shared(q, kc, vc, sc, pre, i32_790, cu_req, table, lens, cu)
        return (o, *lib.sample_logits(o.float().flatten(1) @ head, u, temperature=temp, top_p=temp))

    i32_790, cu_req = i32(790), i32(0, T)
    step(fused, u)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(fused, u)
    for i in range(3):
        fused.copy_(torch.randn_like(fused))
        u.copy_(torch.rand_like(u))
        g.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in got]
        cache = kc.clone(), vc.clone(), sc.clone()
        want = step(fused, u)
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
        for a, b in zip(cache, (kc, vc, sc)):
            assert torch.equal(a, b)


def test_example_draws_tokens(ex, capsys):
    ex.main()
    assert "drawn with" in capsys.readouterr().out
