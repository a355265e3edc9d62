"""One decoder layer of a serving loop on the library's operators.

    python examples/decode_layer.py

A step of M rows (one token of each of several requests, a prompt's piece, or
the drafts of a speculative tree) goes through

    rmsnorm_residual        -> bf16 rows
    qgemm_w4a16_skinny      -> q, k, v (fp32)
    (rotary embedding, torch)
    kv8_block_plan          -> pages and slots of the step's tokens
    kv8_append              -> keys and values into the paged 8-bit cache
    attn_kv8_paged          -> attention of the step's rows over the cache
    qgemm_w4a16_skinny      -> output projection
    rmsnorm_residual_i8     -> int8 rows after the randomized Hadamard transform
    gemm_w8a8_i32           -> gate and up
    (SwiGLU, torch)
    qgemm_w4a16_skinny      -> down projection, the next layer's input

Weights are random; the point is how the calls fit together: all lengths,
tables and slots stay on the GPU, and rejected drafts are given back by a plan
with smaller lengths. (Accepted drafts that are not the first ones of their
tree are appended again in their order after such a plan.)
"""
from __future__ import annotations

import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import skinny_gemm_qgemv_gb300 as lib  # noqa: E402
import synth  # noqa: E402


def rotate(x, positions, base=10000.0):
    """Rotary embedding of x fp32 [M][heads][D] at positions int32 [M] (angles in float64: far positions)."""
    D = x.shape[-1]
    freq = base ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    angle = positions.clamp(min=0).double()[:, None] * freq
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)


class PagedCache:
    """Blocks of one layer's 8-bit cache and the requests' block lists, all on the GPU."""

    def __init__(self, requests, num_blocks, max_blocks, Hkv, D, block_size=16, dtype=torch.int8, device="cuda"):
        shape = (num_blocks, Hkv, block_size, D)
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        self.scales = torch.zeros((num_blocks, Hkv, 2), device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((requests, max_blocks), -1, **i32)
        self.free = torch.arange(num_blocks, **i32)
        self.count = torch.tensor([num_blocks], **i32)
        self.lens = torch.zeros(requests, **i32)
        self.block_size = block_size

    def resize(self, new_lens, max_tokens):
        """Grow or shrink the requests to new_lens: (cu_new, slots, positions, info) of the new tokens. A plan that is
        refused (info[3] is not 0: too few blocks, say) changes nothing, so the lengths stay as they were too."""
        out = lib.kv8_block_plan(self.lens, new_lens, self.table, self.free, self.count, self.block_size, max_tokens,
                                 free_count_out=self.count)
        self.lens = torch.where(out[4][3:] == 0, new_lens, self.lens)
        return out[1:]


class DecodeLayer:
    def __init__(self, hidden=1024, heads=8, kv_heads=2, head_dim=128, intermediate=2048, seed=0, device="cuda"):
        self.heads, self.kv_heads, self.head_dim, self.device = heads, kv_heads, head_dim, device
        w4 = lambda n, k, slot: synth.w4_weights(n, k, seed=seed, slot=slot, device=device)  # noqa: E731
        self.wq, self.wk, self.wv = (w4(h * head_dim, hidden, s) for h, s in ((heads, 0), (kv_heads, 1), (kv_heads, 2)))
        self.wo = w4(hidden, heads * head_dim, 3)
        self.wdown = w4(hidden, intermediate, 4)
        self.norm1 = 1 + synth.normal_f32((hidden,), 0.1, seed, 5, device)
        self.norm2 = 1 + synth.normal_f32((hidden,), 0.1, seed, 6, device)
        self.sign_bits = synth.sign_bits(hidden, seed, 7).to(device)
        # gate and up as one int8 matrix, its rows transformed and quantized like the activations
        w = synth.normal_f32((2 * intermediate, hidden), 0.02, seed, 8, device).to(torch.bfloat16)
        self.w8, self.s8 = lib.hadamard32_quant_i8(w, self.sign_bits)

    def step(self, x, residual, cache, new_lens, tree=None):
        """x, residual fp32 [M][hidden]: the last layer's output and the residual stream (updated in place). Returns
        this layer's output and everything in between by name. Where the plan was refused (t["info"][3] is not 0) nothing
        was stored and no row attended: the output and the residual stream of that step are to be dropped."""
        M = x.shape[0]
        t = dict(x=x, old_residual=residual.clone())
        t["h1"], _ = lib.rmsnorm_residual(x, self.norm1, residual=residual, residual_out=residual)
        q, k, v = (lib.qgemm_w4a16_skinny(*w, t["h1"]).unflatten(1, (-1, self.head_dim))
                   for w in (self.wq, self.wk, self.wv))
        t["cu"], t["slots"], t["positions"], t["info"] = cache.resize(new_lens, M)
        t["q"] = rotate(q, t["positions"]).to(torch.bfloat16)
        t["k"], t["v"] = rotate(k, t["positions"]), v
        lib.kv8_append(t["k"], t["v"], t["slots"], cache.k, cache.v, cache.scales)
        t["attn"] = lib.attn_kv8_paged(t["q"], cache.k, cache.v, cache.scales, cache.table, cache.lens, t["cu"],
                                       tree_mask=tree)
        t["o"] = lib.qgemm_w4a16_skinny(*self.wo, t["attn"].flatten(1))
        t["residual1"] = residual.clone()
        t["h8"], t["s"], _ = lib.rmsnorm_residual_i8(t["o"], self.norm2, residual=residual, sign_bits=self.sign_bits,
                                                     residual_out=residual)
        c = lib.gemm_w8a8_i32(t["h8"], self.w8)
        gu = c.float() * (t["s"][:, None] * self.s8[None, :] / 32)
        gate, up = gu.chunk(2, 1)
        t["act"] = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16).contiguous()
        t["y"] = lib.qgemm_w4a16_skinny(*self.wdown, t["act"])
        return t["y"], t


def tree_words(parents, device="cuda"):
    """Mask words of a draft tree: draft i sees itself and its ancestors (parents[i] < i, -1: the context only)."""
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    words = [w - (1 << 32) if w >> 31 else w for w in words]
    return torch.tensor(words, dtype=torch.int32, device=device)


def main():
    torch.manual_seed(0)
    R, hidden = 4, 1024
    layer = DecodeLayer(hidden)
    cache = PagedCache(R, num_blocks=256, max_blocks=64, Hkv=layer.kv_heads, D=layer.head_dim)
    lens = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731

    def rows(m):
        return torch.randn(m, hidden, device="cuda"), torch.randn(m, hidden, device="cuda")

    # prompts of 5, 7, 9 and 11 tokens as one step of 32 rows
    y, t = layer.step(*rows(32), cache, lens(5, 7, 9, 11))
    info = t["info"].tolist()
    assert info[3] == 0, "the plan was refused"           # read once here; a server looks at it where it samples
    print("prompts:", info, "output", tuple(y.shape))
    # decode: one token of every request
    n = [5, 7, 9, 11]
    for _ in range(3):
        n = [a + 1 for a in n]
        y, t = layer.step(*rows(R), cache, lens(*n))
    # speculative verification: six drafts of a tree for every request, its first two accepted (one below the other)
    parents = [-1, 0, 0, 1, 2, 4]
    words = tree_words(parents).repeat(R)
    y, t = layer.step(*rows(6 * R), cache, lens(*[a + 6 for a in n]), tree=words)
    cu, slots, _, info = cache.resize(lens(*[a + 2 for a in n]), 1)
    print("after the rollback:", info.tolist(), "lengths", cache.lens.tolist(), "free blocks", cache.count.item())
    n = [a + 2 for a in n]
    torch.cuda.synchronize()
    began, steps = time.perf_counter(), 50
    for _ in range(steps):
        n = [a + 1 for a in n]
        y, t = layer.step(*rows(R), cache, lens(*n))
    torch.cuda.synchronize()
    print(f"{(time.perf_counter() - began) / steps * 1e6:.0f} us a layer step of {R} requests, contexts", n)
    assert torch.isfinite(y).all() and lib.device_error() == 0


if __name__ == "__main__":
    main()
