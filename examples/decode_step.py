"""A server's steps over a block-quantized cache, from the requests' lengths to their next tokens, through the library's
calls: prompts, then single tokens, each attending over the pages of the cache that are chosen for it.

  qmm_cache_plan (pages, slots, rows)                                                     once a step
  qmm_norm_mx4 -> qmm_mx4_matmul -> qmm_cache_write -> qmm_cache_bounds -> qmm_cache_select
    -> qmm_cache_attend_chosen -> qmm_mx4_linear -> qmm_norm_mx4 -> qmm_mx4_matmul          once a layer
  qmm_norm_q8 -> qmm_matmul -> qmm_sample                                                    once a step

Run as a program it takes four requests through their prompts and a few single tokens, compares what the calls give with plain
torch operations on the same inputs, then captures the step of single tokens as a graph, whose replays carry the
requests on by themselves, and compares their tokens with those of the steps before.

    python examples/decode_step.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_matmul_gb300 as qmm  # noqa: E402

BF16 = torch.bfloat16
EPS = 1e-6


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def mx4_weight(w):
    n, k = w.shape
    codes = torch.empty(qmm.mx4_codes_size(n, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(n, k), dtype=torch.uint8, device="cuda")
    qmm.qmm_mx4_quantize("f32", w, n, k, k, codes, scales)
    return codes, scales


class Layer:
    """One layer's weights and caches: attention, then one product in the place of a feed-forward block."""

    def __init__(self, gen, m):
        def normal(*shape, of=1.0):
            return of * torch.randn(*shape, generator=gen, device="cuda")

        w, q = m.width, m.heads * m.d
        self.qkv = mx4_weight(normal(q + 2 * m.kv_heads * m.d, w, of=1 / math.sqrt(w)))
        self.out = mx4_weight(normal(w, q, of=1 / math.sqrt(q)))
        self.ff = mx4_weight(normal(w, w, of=1 / math.sqrt(w)))
        self.norms = [1 + normal(w, of=0.1) for _ in range(4)]        # before the attention, behind it, before the product, behind it
        size = m.n_pages * qmm.cache_page_size(m.type, m.kv_heads, m.d, m.page)
        self.k_cache, self.v_cache = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.bounds = torch.zeros(m.n_pages * qmm.cache_bounds_size(m.kv_heads, m.d), dtype=torch.uint8, device="cuda")


class Server:
    def __init__(self, seqs=4, layers=2, width=512, heads=8, kv_heads=2, d=64, vocab=1000, page=16, ld_pages=12, n_pages=44, type_="q8_0", budget=5, seed=0):
        self.seqs, self.width, self.heads, self.kv_heads, self.d, self.vocab = seqs, width, heads, kv_heads, d, vocab
        self.page, self.ld_pages, self.n_pages, self.type, self.budget = page, ld_pages, n_pages, type_, budget
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn(vocab, width, generator=gen, device="cuda").to(BF16)
        self.layers = [Layer(gen, self) for _ in range(layers)]
        self.last_norm = 1 + 0.1 * torch.randn(width, generator=gen, device="cuda")
        head = torch.randn(vocab, width, generator=gen, device="cuda") / math.sqrt(width) * 3
        flat = torch.empty(qmm.flat_size("q8_0", width, vocab), dtype=torch.uint8, device="cuda")
        self.head = torch.empty(qmm.tiled_size("q8_0", width, vocab), dtype=torch.uint8, device="cuda")
        qmm.qmm_quantize_weight("q8_0", head, vocab, width, width, flat)
        qmm.qmm_repack("q8_0", flat, width, vocab, self.head)
        # the requests: nothing cached, all pages free
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.pages = torch.full((seqs, ld_pages), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        self.ring_at = torch.tensor([0, n_pages], dtype=torch.int64, device="cuda")
        self.temperature, self.top_p = (torch.full((seqs,), x, device="cuda") for x in (0.9, 0.95))
        self.top_k = int32([40, 0, 5, 1][:seqs] + [0] * (seqs - 4))

    def step(self, tokens, news, u, max_new, max_len, seen=None):
        """One step: `tokens` are the rows' tokens (news[s] of sequence s); returns each sequence's next token.  `seen`, a list, is
        given what the calls read and wrote, layer by layer."""
        n, t, w, hk, d, hq = self.seqs, tokens.shape[0], self.width, self.kv_heads, self.d, self.heads
        q_starts, kv_lens = torch.empty(n + 1, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        slots = torch.empty(t, dtype=torch.int64, device="cuda")
        qmm.qmm_cache_plan(self.lens, news, n, self.page, self.pages, self.ld_pages, self.ring, self.n_pages, self.ring_at, t, q_starts, kv_lens,
                           slots, None, self.lens, self.ring_at)
        h = self.embedding.index_select(0, tokens)                     # the residual stream
        x, post = None, None                                           # the block's output that is still to be added to it, its norm
        codes = torch.empty(t, w // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(qmm.mx4_scales_size(t, w), dtype=torch.uint8, device="cuda")
        need = max(qmm.cache_select_workspace_size(t, hk, self.page, max_len),
                   qmm.cache_attend_chosen_workspace_size(t, hk, hq, d, self.page, self.budget), qmm.mx4_linear_workspace_size(t, hq * d))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def norm(x, post, weight):
            """The stream with x added, and its norm as an operand."""
            out = torch.empty_like(h)
            qmm.qmm_norm_mx4("bf16", x, w, "bf16", h, w, t, w, post, None, 0, 1.0, weight, EPS, out, w, codes, scales)
            return out

        def product(weight, rows):
            y = torch.empty(t, rows, dtype=BF16, device="cuda")
            qmm.qmm_mx4_matmul(*weight, w, rows, codes, scales, t, "bf16", y, rows)
            return y

        for layer in self.layers:
            before = (h, x, post)
            h = norm(x, post, layer.norms[0])
            qkv = product(layer.qkv, (hq + 2 * hk) * d)
            ld = qkv.stride(0)
            q, k, v = qkv[:, : hq * d], qkv[:, hq * d : (hq + hk) * d], qkv[:, (hq + hk) * d :]
            qmm.qmm_cache_write(self.type, "bf16", k, v, ld, ld, t, hk, d, slots, layer.k_cache, layer.v_cache, self.n_pages, self.page)
            qmm.qmm_cache_bounds(self.type, layer.k_cache, self.n_pages, self.page, hk, d, self.pages, self.ld_pages, q_starts, kv_lens, n, t, max_new,
                                 layer.bounds)
            chosen = torch.full((t, hk, self.budget), -1, dtype=torch.int32, device="cuda")
            qmm.qmm_cache_select(layer.bounds, self.n_pages, self.page, hk, d, self.pages, self.ld_pages, q_starts, kv_lens, n, "bf16", q, ld, t, hq, None,
                                 max_new, max_len, 1, 2, self.budget, chosen, ws, need)
            o = torch.empty(t, hq * d, dtype=BF16, device="cuda")
            qmm.qmm_cache_attend_chosen(self.type, layer.k_cache, layer.v_cache, self.n_pages, self.page, hk, d, self.pages, self.ld_pages, q_starts,
                                        kv_lens, n, "bf16", q, ld, t, hq, None, 1 / math.sqrt(d), chosen, self.budget, o, hq * d, None, ws, need)
            x = torch.empty(t, w, dtype=BF16, device="cuda")
            qmm.qmm_mx4_linear(*layer.out, hq * d, w, "bf16", o, hq * d, t, "bf16", x, w, ws, need)
            if seen is not None:
                seen.append({"before": before, "h": h, "q": q, "chosen": chosen, "o": o, "q_starts": q_starts, "kv_lens": kv_lens, "slots": slots})
            h = norm(x, layer.norms[1], layer.norms[2])
            x, post = product(layer.ff, w), layer.norms[3]
        # logits of each sequence's last row
        last = (q_starts[1:] - 1).clamp(min=0).long()
        a_q, a_d = torch.empty(t, w, dtype=torch.int8, device="cuda"), torch.empty(t, w // 32, dtype=torch.float16, device="cuda")
        qmm.qmm_norm_q8("bf16", x, w, "bf16", h, w, t, w, post, None, 0, 1.0, self.last_norm, EPS, torch.empty_like(h), w, a_q, a_d)
        a_q, a_d = a_q.index_select(0, last), a_d.index_select(0, last)
        logits = torch.empty(n, self.vocab, device="cuda")
        qmm.qmm_matmul("q8_0", self.head, w, self.vocab, a_q, a_d, n, logits, self.vocab)
        out, logp = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
        qmm.qmm_sample("f32", logits, self.vocab, n, self.vocab, self.temperature, self.top_k, self.top_p, None, u, out, logp)
        if seen is not None:
            seen.append({"logits": logits, "u": u, "tokens": out, "logp": logp})
        return out

    def cached(self, layer, starts, total):
        """The cached keys and values of all sequences in fp64."""
        k, v = (torch.empty(total, self.kv_heads * self.d, device="cuda") for _ in range(2))
        ld = self.kv_heads * self.d
        qmm.qmm_cache_read(self.type, layer.k_cache, layer.v_cache, self.n_pages, self.page, self.kv_heads, self.d, self.pages, self.ld_pages, starts,
                           self.seqs, total, "f32", k, v, ld, ld)
        return (a.view(total, self.kv_heads, self.d).double() for a in (k, v))


def check(server, seen, lens, news):
    """The calls of one step against plain operations in 64 bits on what they read."""
    page, g, d = server.page, server.heads // server.kv_heads, server.d
    starts = [sum(lens[:s]) for s in range(len(lens) + 1)]
    for layer, got in zip(server.layers, seen):
        # the plan: every row's slot lies on its own page, and the stream holds what the norms' formula says
        assert got["kv_lens"].tolist() == lens and len(set(got["slots"].tolist())) == sum(news)
        h, x, post = got["before"]
        want = h.double()
        if x is not None:
            b = x.double()
            want = want + b * torch.rsqrt(b.pow(2).mean(1, keepdim=True) + EPS) * post.double()
        assert ((got["h"].double() - want).abs() <= 2.0 ** -7 * (want.abs() + h.double().abs()) + 1e-6).all()
        k, v = server.cached(layer, int32(starts), starts[-1])
        row = 0
        for s, (n, new) in enumerate(zip(lens, news)):
            for i in range(new):
                place = n - new + i
                for head in range(server.kv_heads):
                    pages = [p for p in got["chosen"][row, head].tolist() if p >= 0]
                    own = place // page
                    assert pages == sorted(set(pages)) and pages[0] == 0 and pages[-1] == own and max(0, own - 1) in pages
                    assert len(pages) == min(server.budget, own + 1)
                    keys = torch.tensor([j for p in pages for j in range(p * page, min(place + 1, p * page + page))], device="cuda") + starts[s]
                    q = got["q"][row].view(server.heads, d)[head * g : head * g + g].double()
                    w = torch.softmax(q @ k[keys, head].t() / math.sqrt(d), -1)
                    want = w @ v[keys, head]
                    o = got["o"][row].view(server.heads, d)[head * g : head * g + g].double()
                    assert ((o - want).abs() <= 2.0 ** -6 * want.abs().amax() + 1e-6).all()
                row += 1
    end = seen[-1]
    z = end["logits"].double()
    for s in range(server.seqs):
        order = torch.argsort(-z[s], stable=True)
        w = torch.exp((z[s] - z[s].max()) / float(server.temperature[s]))
        k = int(server.top_k[s])
        order = order[: k if k > 0 else server.vocab]
        before = torch.cumsum(w[order], 0) - w[order]
        kept = order[: max(1, int((before < float(server.top_p[s]) * w[order].sum()).sum()))].sort().values
        upto = torch.cumsum(w[kept], 0) / w[kept].sum()
        u = float(end["u"][s])
        if float((upto - u).abs().min()) > 1e-6:
            assert int(end["tokens"][s]) == int(kept[int((upto <= u).sum())])


def main(prompts=(70, 3, 33, 100), steps=30, type_="q8_0", seed=0):
    server = Server(len(prompts), type_=type_, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    max_len = server.ld_pages * server.page
    tokens = torch.randint(0, server.vocab, (sum(prompts),), generator=gen, device="cuda", dtype=torch.int32)
    us = torch.rand(steps + 1, len(prompts), generator=gen, device="cuda")
    lens, seen = list(prompts), []
    tokens = server.step(tokens, int32(prompts), us[0], max(prompts), max_len, seen)
    check(server, seen, lens, list(prompts))
    ones = torch.ones(len(prompts), dtype=torch.int32, device="cuda")
    state = [a.clone() for a in (server.lens, server.pages, server.ring, server.ring_at)]
    caches = [[a.clone() for a in (x.k_cache, x.v_cache, x.bounds)] for x in server.layers]
    first, eager = tokens.clone(), []
    for i in range(steps):
        seen = []
        tokens = server.step(tokens, ones, us[i + 1], 1, max_len, seen)
        eager.append(tokens.tolist())
        lens = [x + 1 for x in lens]
        if i % 10 == 9:
            check(server, seen, lens, [1] * len(lens))
    # the same steps as replays of one graph
    for a, b in zip((server.lens, server.pages, server.ring, server.ring_at), state):
        a.copy_(b)
    for layer, kept in zip(server.layers, caches):
        for a, b in zip((layer.k_cache, layer.v_cache, layer.bounds), kept):
            a.copy_(b)
    now, u = first.clone(), us[1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now.copy_(server.step(now, ones, u, 1, max_len))
    replayed = []
    for i in range(steps):
        u.copy_(us[i + 1])
        graph.replay()
        replayed.append(now.tolist())
    assert replayed == eager
    torch.cuda.synchronize()
    assert qmm.qmm_device_status() == 0
    return lens, eager


if __name__ == "__main__":
    for t in ("q8_0", "q4_0"):
        lens, tokens = main(type_=t)
        print(f"{t}: tokens cached {lens}, {len(tokens)} steps, eager and replayed alike")
