"""The attention half of a decoder layer on 4-bit weights and a block-quantized cache: a prompt, then trees of
drafted tokens, through the library's calls.

  x -> qmm_mx4_linear (one weight for queries, keys and values) -> qmm_cache_write -> qmm_cache_attend
    -> qmm_mx4_linear (output projection)

Run as a program it takes two sequences through a prompt and one step of drafted trees, and compares every
result with the same layer in plain torch operations (fp32, weights and activations at their MX4 values, keys
and values at their cached values).

    python examples/mx4_attention_layer.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_matmul_gb300 as qmm  # noqa: E402

BF16 = torch.bfloat16


class Mx4Linear:
    """y = MX4(x) @ MX4(w)^T, bf16 rows in and out."""

    def __init__(self, w: torch.Tensor):
        self.n, self.k = w.shape
        self.codes = torch.empty(qmm.mx4_codes_size(self.n, self.k), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(qmm.mx4_scales_size(self.n, self.k), dtype=torch.uint8, device="cuda")
        qmm.qmm_mx4_quantize("f32", w, self.n, self.k, self.k, self.codes, self.scales)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        m = x.shape[0]
        y = torch.empty(m, self.n, dtype=BF16, device="cuda")
        need = qmm.mx4_linear_workspace_size(m, self.k)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        qmm.qmm_mx4_linear(self.codes, self.scales, self.k, self.n, "bf16", x, x.stride(0), m, "bf16", y, self.n, ws, need)
        return y


class AttentionLayer:
    """Projections and a paged cache of one layer; `type_` is the cache's block type (q8_0 or q4_0)."""

    def __init__(self, w_qkv, w_out, heads: int, kv_heads: int, d: int, type_="q8_0", page=64, n_pages=64):
        self.qkv, self.out = Mx4Linear(w_qkv), Mx4Linear(w_out)
        self.heads, self.kv_heads, self.d, self.type, self.page, self.n_pages = heads, kv_heads, d, type_, page, n_pages
        size = qmm.cache_page_size(type_, kv_heads, d, page)
        self.k_cache, self.v_cache = (torch.zeros(n_pages * size, dtype=torch.uint8, device="cuda") for _ in range(2))

    def slots(self, table, seq_of, pos):
        """Slot of each token: its sequence's page, and its place there."""
        return table[seq_of, pos // self.page].long() * self.page + pos % self.page

    def step(self, x, table, q_starts, kv_lens, slots, tree, max_new: int, max_len: int):
        """New tokens of all sequences (rows q_starts[s].. of x), whose places in the cache are `slots`; kv_lens
        counts them in.  tree: a word per token saying which new tokens it sees, or None for a prompt."""
        t, (h, hk, d) = x.shape[0], (self.heads, self.kv_heads, self.d)
        qkv = self.qkv(x)
        q, k, v = qkv[:, : h * d], qkv[:, h * d : (h + hk) * d], qkv[:, (h + hk) * d :]
        ld = qkv.stride(0)
        qmm.qmm_cache_write(self.type, "bf16", k, v, ld, ld, t, hk, d, slots, self.k_cache, self.v_cache, self.n_pages, self.page)
        o = torch.empty(t, h * d, dtype=BF16, device="cuda")
        need = qmm.cache_attend_workspace_size(kv_lens.shape[0], max_new, hk, h, d, max_len)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        qmm.qmm_cache_attend(self.type, self.k_cache, self.v_cache, self.n_pages, self.page, hk, d, table, table.shape[1], q_starts,
                             kv_lens, kv_lens.shape[0], "bf16", q, ld, t, h, tree, 1 / math.sqrt(d), max_new, max_len, o, h * d, None,
                             ws, need)
        return self.out(o), q, o

    def cached(self, table, starts, total: int):
        """The cached keys and values of all sequences, as fp32 rows."""
        hk, d = self.kv_heads, self.d
        k, v = (torch.empty(total, hk * d, device="cuda") for _ in range(2))
        qmm.qmm_cache_read(self.type, self.k_cache, self.v_cache, self.n_pages, self.page, hk, d, table, table.shape[1], starts,
                           starts.shape[0] - 1, total, "f32", k, v, hk * d, hk * d)
        return k.view(total, hk, d), v.view(total, hk, d)


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def mx4_values(x: torch.Tensor) -> torch.Tensor:
    """fp32 rows at their MX4 values, by the library's converters."""
    r, k = x.shape
    x = x.float().contiguous()
    codes = torch.empty(qmm.mx4_codes_size(r, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(r, k), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    qmm.qmm_mx4_quantize("f32", x, r, k, k, codes, scales)
    qmm.qmm_mx4_dequantize(codes, scales, r, k, "f32", y, k)
    return y


def plain_attention(q, k, v, seen, scale):
    """q [n, h, d], k and v [l, hk, d], seen [n, l] -> [n, h, d], in fp64."""
    g = q.shape[1] // k.shape[1]
    k, v = (a.double().repeat_interleave(g, 1) for a in (k, v))
    s = torch.einsum("nhd,lhd->nhl", q.double(), k) * scale
    p = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), -1)
    return torch.einsum("nhl,lhd->nhd", p, v)


def close(a, b, what):
    """bf16 results: a few roundings of 2^-9 of the row's size."""
    err = (a.double() - b.double()).abs()
    tol = 2.0 ** -6 * b.double().abs().amax(-1, keepdim=True) + 1e-6
    assert (err <= tol).all(), f"{what}: {float(err.max())}"


def main(type_="q8_0", width=1024, heads=8, kv_heads=2, d=64, prompts=(100, 37), drafts=(6, 4), seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w_qkv = torch.randn((heads + 2 * kv_heads) * d, width, generator=gen, device="cuda") / math.sqrt(width)
    w_out = torch.randn(width, heads * d, generator=gen, device="cuda") / math.sqrt(heads * d)
    layer = AttentionLayer(w_qkv, w_out, heads, kv_heads, d, type_)
    n = len(prompts)
    table = torch.arange(4 * n, dtype=torch.int32, device="cuda").view(n, 4).flip(0).contiguous()   # four pages each
    trees = [[1 << i | (0 if i == 0 else 1) | (1 << i // 2 if i > 1 else 0) for i in range(c)] for c in drafts]
    done = [0] * n
    for counts, words in ((prompts, None), (drafts, trees)):
        seq_of = torch.cat([torch.full((c,), s, device="cuda") for s, c in enumerate(counts)])
        pos = torch.cat([torch.arange(done[s], done[s] + c, device="cuda") for s, c in enumerate(counts)])
        lens = [a + c for a, c in zip(done, counts)]
        q_starts = [sum(counts[:s]) for s in range(n + 1)]
        x = torch.randn(sum(counts), width, generator=gen, device="cuda").to(BF16)
        tree = None if words is None else torch.tensor(sum(words, []), dtype=torch.int64, device="cuda")
        y, q, o = layer.step(x, table, int32(q_starts), int32(lens), layer.slots(table, seq_of, pos), tree, max(counts), max(lens))
        # the same step in plain operations, from the library's q and the cached keys and values
        close(q, (mx4_values(x) @ mx4_values(w_qkv).t())[:, : heads * d], "projection")
        k, v = layer.cached(table, int32([sum(lens[:s]) for s in range(n + 1)]), sum(lens))
        for s, c in enumerate(counts):
            rows, keys = slice(q_starts[s], q_starts[s] + c), slice(sum(lens[:s]), sum(lens[: s + 1]))
            seen = torch.ones(c, lens[s], dtype=torch.bool, device="cuda")
            for i in range(c):
                for j in range(c):
                    seen[i, done[s] + j] = j <= i if words is None else bool(words[s][i] >> j & 1)
            ref = plain_attention(q[rows].view(c, heads, d), k[keys], v[keys], seen, 1 / math.sqrt(d))
            close(o[rows], ref.reshape(c, -1), "attention")
        close(y, mx4_values(o) @ mx4_values(w_out).t(), "output")
        done = lens
    torch.cuda.synchronize()
    assert qmm.qmm_device_status() == 0
    return done


if __name__ == "__main__":
    for t in ("q8_0", "q4_0"):
        print(f"{t}: tokens cached {main(t)}, every step as in plain operations")
