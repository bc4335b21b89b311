"""The operators of a decoder step around its products and its cache, as cases to be measured.

  plan     page tables, slots and row starts of a step, from the requests' lengths and new tokens
  bounds   for each page of cached keys the range of its keys, which the choice of pages reads
  sparse   attention of new tokens over the pages of the cache that a cheap score chooses for each token and key/value head
  norm     the norm behind a block, its gate and residual, and the norm before the next one
  sample   tokens from logits with temperature, top-k, top-p and min-p

With `own` false, run() computes each in elementary torch operations; with `own` true it makes the library's calls.
exact() computes them in fp64.  Where a rule fixes fp32 steps (block scales and codes, the scores that pages are
chosen by), both follow it.

Layouts (both sides read and write the same buffers):
  Cache page of P tokens: for each head [P][D] codes (q8_0: int8; q4_0: [P][D/2] bytes, byte j of a block of 32
    holds element j low and j + 16 high), then [P][D/32] fp16 scales.
  Bounds of a page: for each head [2][D] int8 codes (lowest, highest), [D/32] fp16 scales, zeros up to 16 bytes.
  Ring of free pages: int32 [n], with two counters: entries first..last - 1 (modulo n) are free.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
WORKSPACE = 128 << 20   # bytes a server keeps for scores and partial results


def listed():
    return [
        # a decode step of a small batch: one new token each, a page more now and then
        {"name": "plan decode step", "op": "plan", "seqs": 64, "prompts": 0, "new": 1, "hi": 8192, "page": 64, "free": 1.0},
        # a step of a large server: most requests decode, some bring prompts, some are idle, done or have to wait
        {"name": "plan mixed step", "op": "plan", "seqs": 2048, "prompts": 100, "new": 8192, "hi": 32768, "page": 16, "free": 0.7},
        # a decode step: the pages with the new tokens
        {"name": "bounds decode step", "op": "bounds", "type": "q8_0", "seqs": 64, "lo": 0, "hi": 500, "new": 1, "heads": 8, "d": 128, "page": 64},
        # four prompts, just written
        {"name": "bounds prompts", "op": "bounds", "type": "q4_0", "seqs": 4, "lo": 3000, "hi": 16384, "new": 16384, "heads": 8, "d": 128, "page": 64},
        # one token of one long conversation: latency
        {"name": "sparse one token", "op": "sparse", "type": "q8_0", "seqs": 1, "lo": 131071, "hi": 131071, "new": 1, "tree": False, "heads": 8, "group": 4, "d": 128, "page": 64, "sinks": 1, "recent": 4, "budget": 32, "dtype": "bf16"},
        # a decode step of ragged sequences, an empty one and ones shorter than the budget among them
        {"name": "sparse batch", "op": "sparse", "type": "q8_0", "seqs": 32, "lo": 0, "hi": 32768, "new": 1, "tree": False, "heads": 8, "group": 4, "d": 128, "page": 64, "sinks": 1, "recent": 4, "budget": 64, "dtype": "bf16"},
        # a piece of a long prompt
        {"name": "sparse prompt piece", "op": "sparse", "type": "q4_0", "seqs": 1, "lo": 65536, "hi": 65536, "new": 128, "tree": False, "heads": 8, "group": 4, "d": 128, "page": 64, "sinks": 1, "recent": 2, "budget": 32, "dtype": "f16"},
        # between two blocks in a decode step: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "n": 4096, "x": "bf16", "h": "bf16", "form": "bf16", "post": False, "gate": "none"},
        # between two blocks of a prompt, with both norms and a gate for each channel
        {"name": "norm prompt", "op": "norm", "rows": 8192, "n": 4096, "x": "bf16", "h": "bf16", "form": "bf16", "post": True, "gate": "all"},
        # the next token of one request, from the logits of the output product
        {"name": "sample one request", "op": "sample", "rows": 1, "v": 128256, "dtype": "f32", "mode": "chat"},
        # a batch whose requests ask for different things, greedy ones among them
        {"name": "sample mixed batch", "op": "sample", "rows": 64, "v": 128256, "dtype": "bf16", "mode": "mixed"},
        # a large batch with nothing but a temperature: every logit counts
        {"name": "sample rollouts", "op": "sample", "rows": 256, "v": 128256, "dtype": "f32", "mode": "all"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "bounds", "sparse", "sparse", "norm", "norm", "sample", "sample"])
    if op == "plan":
        return {"op": op, "seqs": _log(rng, 1, 2048), "prompts": _log(rng, 1, 100) - 1, "new": _log(rng, 1, 8192), "hi": _log(rng, 20, 32768),
                "page": rng.choice([16, 32, 64, 128, 256]), "free": rng.choice([1.0, 1.0, rng.random()])}
    if op == "norm":
        n = 32 * _log(rng, 1, 512)
        form = rng.choice(["f32", "f16", "bf16", "q8", "mx4"])
        if form not in ("q8", "mx4") and rng.random() < 0.3:
            n += rng.randrange(1, 32)
        return {"op": op, "rows": _log(rng, 1, max(1, min(8192, (1 << 25) // n))), "n": n, "x": rng.choice(["f32", "f16", "bf16"]),
                "h": rng.choice(["f32", "bf16"]), "form": form, "post": rng.random() < 0.5, "gate": rng.choice(["none", "all", "rows"])}
    if op == "sample":
        v = _log(rng, 1000, 200000)
        return {"op": op, "rows": _log(rng, 1, min(256, (1 << 25) // v)), "v": v, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "mode": rng.choice(["chat", "mixed", "mixed", "all"])}
    c = {"op": op, "type": rng.choice(["q8_0", "q4_0"]), "seqs": _log(rng, 1, 48), "heads": rng.choice([1, 2, 4, 8]),
         "d": rng.choice([64, 96, 128, 256]), "page": rng.choice([16, 32, 64, 128])}
    most = min(131072, (1 << 27) // (c["seqs"] * c["heads"] * c["d"]))
    if op == "bounds":
        c["hi"] = _log(rng, 20, max(20, most // 2))
        c["lo"] = rng.randrange(0, c["hi"] + 1)
        return c | {"new": rng.choice([1, _log(rng, 1, c["hi"])])}
    tree = rng.random() < 0.3
    c |= {"new": rng.randrange(2, 33) if tree else rng.choice([1, 1, rng.randrange(2, 17)]), "tree": tree, "group": rng.choice([1, 2, 3, 4, 7, 8, 16]),
          "sinks": rng.choice([0, 1, 2]), "recent": rng.randrange(1, 5), "dtype": rng.choice(["f16", "bf16"])}
    # the chosen pages of all tokens and heads, as the plain form gathers them
    c["budget"] = max(10, min(_log(rng, 10, 128), (1 << 28) // (c["seqs"] * c["new"] * c["heads"] * c["page"] * c["d"])))
    c["seqs"] = max(1, min(c["seqs"], (1 << 28) // (c["budget"] * c["new"] * c["heads"] * c["page"] * c["d"])))
    # and the scores of all pages
    rows = c["seqs"] * c["new"] * c["heads"] * c["group"] * (c["d"] // 32)
    c["hi"] = _log(rng, 500, max(500, min(most, c["page"] * (1 << 25) // rows)))
    c["lo"] = rng.randrange(0, c["hi"] + 1)
    return c


# ------------------------------------------------------------------------------------------- sizes
def _lens(case):
    """The sequences' lengths: spread from lo to hi, in a fixed odd order."""
    n, lo, hi = case["seqs"], case.get("lo", 0), case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * ((i * 7919 + n // 2) % n) // (n - 1) for i in range(n)]


def _news(case):
    if case["op"] != "plan":
        return [min(n, case["new"]) for n in _lens(case)]
    # one token each; the prompts, at fixed odd places, bring up to `new`; a few requests are idle (0) or done (-1)
    rng = random.Random(case["seqs"] * 31 + case["new"])
    out = [rng.choice([1] * 20 + [0, -1]) if case["seqs"] > 64 else 1 for _ in range(case["seqs"])]
    for i in rng.sample(range(case["seqs"]), min(case["prompts"], case["seqs"])):
        out[i] = rng.randrange(1, case["new"] + 1)
    return out


def _plan_lens(case):
    """Cached before the step: a prompt's request has nothing yet, or a first piece of it."""
    return [n // 4 if new > 1 else n for n, new in zip(_lens(case), _news(case))]


def _up(a, b):
    return -(-a // b)


def _code_bytes(t, d):
    return d if t == "q8_0" else d // 2


def _token_bytes(t, d):
    return _code_bytes(t, d) + d // 32 * 2


def _bound_bytes(d):
    return _up(2 * d + d // 32 * 2, 16) * 16


def _touched(case):
    """(sequence, page number, tokens in it) of the pages that hold new tokens."""
    p = case["page"]
    return [(s, k, min(n - k * p, p)) for s, (n, new) in enumerate(zip(_lens(case), _news(case))) if new for k in range((n - new) // p, (n - 1) // p + 1)]


def work(case):
    op = case["op"]
    if op == "plan":
        lens, news, p = _plan_lens(case), _news(case), case["page"]
        rows = sum(max(0, x) for x in news)
        moved = sum(_up(n + new, p) - _up(n, p) if new >= 0 else _up(n, p) for n, new in zip(lens, news))
        return {"bytes": 20 * len(lens) + 12 * rows + 8 * moved, "flops": 10 * (len(lens) + rows)}
    if op == "norm":
        m, n = case["rows"], case["n"]
        out = {"q8": 34 / 32, "mx4": 17 / 32}.get(case["form"]) or SIZE[case["form"]]
        gate = {"none": 0, "all": 1, "rows": m}[case["gate"]] * n * SIZE[case["x"]]
        return {"bytes": int(m * n * (SIZE[case["x"]] + 2 * SIZE[case["h"]] + out)) + gate + 4 * n * (1 + case["post"]), "flops": 10 * m * n}
    if op == "sample":
        return {"bytes": case["rows"] * (case["v"] * SIZE[case["dtype"]] + 28), "flops": 4 * case["rows"] * case["v"]}
    t, h, d, p = case["type"], case["heads"], case["d"], case["page"]
    if op == "bounds":
        pages = _touched(case)
        return {"bytes": h * (sum(n for _, _, n in pages) * _token_bytes(t, d) + len(pages) * (2 * d + d // 32 * 2)), "flops": 3 * h * d * sum(n for _, _, n in pages)}
    lens, news, g = _lens(case), _news(case), case["group"]
    pages = sum(_up(n, p) for n, new in zip(lens, news) if new)
    rows = sum(news) * h * g
    scored = sum(_up(n, p) * new for n, new in zip(lens, news)) * h * g
    read = sum(min(_up(n, p), case["budget"]) * p * new for n, new in zip(lens, news))
    # a page that several tokens choose is read once
    keys = sum(min(n, min(_up(n, p), case["budget"]) * p * new) for n, new in zip(lens, news))
    return {"bytes": h * (pages * (2 * d + d // 32 * 2) + 2 * keys * _token_bytes(t, d)) + 2 * rows * d * SIZE[case["dtype"]] + 4 * sum(news) * h * case["budget"],
            "flops": 4 * scored * d + 4 * read * h * g * d}


# ------------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    s = [0]
    for c in counts:
        s.append(s[-1] + c)
    return s


def _ancestors(rng, n, chain):
    """For each drafted token of a tree the set of tokens on its way from the root, as bits."""
    bits = []
    for i in range(n):
        up = -1 if i == 0 else i - 1 if chain else rng.randrange(max(-1, i - 8), i)
        bits.append((1 << i) | (bits[up] if up >= 0 else 0))
    return [b - (1 << 64) if b >= 1 << 63 else b for b in bits]


def _prepare_plan(case, s, gen):
    lens, news, p = _plan_lens(case), _news(case), case["page"]
    n, rows = len(lens), sum(max(0, x) for x in news)
    ld = max(1, max(_up(a + max(0, b), p) for a, b in zip(lens, news)))
    held = [_up(a, p) for a in lens]
    need = sum(_up(a + b, p) - _up(a, p) for a, b in zip(lens, news) if b > 0)
    free = int(need * case["free"]) + (3 if case["free"] == 1.0 else 0)
    count = sum(held) + free + 5
    order = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    place = torch.arange(ld, device="cuda")[None, :]
    have = _int32(held)[:, None]
    at = _int32(_starts(held)[:-1])[:, None] + place
    s["pages"] = torch.where(place < have, order[at.clamp(max=count - 1).long()], -1).contiguous()
    first = 7 * count + count // 3                      # the ring has gone round a few times
    s["ring"] = torch.full((count,), -1, dtype=torch.int32, device="cuda")
    s["ring"][(first + torch.arange(free, device="cuda")) % count] = order[sum(held) : sum(held) + free]
    s["ring_at"] = torch.tensor([first, first + free], dtype=torch.int64, device="cuda")
    s["lens"], s["news"], s["rows"] = _int32(lens), _int32(news), rows
    s["q_starts"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    s["kv_lens"], s["next_lens"] = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    s["slots"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
    s["positions"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["next_at"] = torch.zeros(2, dtype=torch.int64, device="cuda")
    return s


def _prepare_norm(case, s, gen):
    m, n, dt = case["rows"], case["n"], DTYPES[case["x"]]
    big = 1 + 9 * (torch.rand(n, generator=gen, device="cuda") < 0.01)      # a few channels of a residual stream are large
    s["x"] = (0.5 * _normal(gen, m, n)).to(dt)
    s["h"] = (2 * _normal(gen, m, n) * big).to(DTYPES[case["h"]])
    s["h_out"] = torch.zeros_like(s["h"])
    s["w_pre"] = 1 + 0.1 * _normal(gen, n)
    s["w_post"] = 1 + 0.1 * _normal(gen, n) if case["post"] else None
    g = {"none": None, "all": (1, n), "rows": (m, n)}[case["gate"]]
    s["gate"] = None if g is None else torch.sigmoid(_normal(gen, *g)).to(dt)
    s["scale"], s["eps"] = 0.75, 1e-6
    if case["form"] == "q8":
        s["a_q"] = torch.zeros(m, n, dtype=torch.int8, device="cuda")
        s["a_d"] = torch.zeros(m, n // 32, dtype=torch.float16, device="cuda")
    elif case["form"] == "mx4":
        s["codes"] = torch.zeros(m, n // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(_up(m, 128) * _up(n, 128) * 512, dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    else:
        s["y"] = torch.zeros(m, n, dtype=DTYPES[case["form"]], device="cuda")
    return s


def _prepare_sample(case, s, gen, seed):
    m, v, rng = case["rows"], case["v"], random.Random(seed)
    # logits of a model that is sure now and then: a wide bulk, and a few candidates that stand out
    z = 2.5 * _normal(gen, m, v)
    some = torch.randint(0, v, (m, 20), generator=gen, device="cuda")
    z.scatter_add_(1, some, 6 + 4 * _normal(gen, m, 20))
    s["logits"] = z.to(DTYPES[case["dtype"]])
    s["u"] = torch.rand(m, generator=gen, device="cuda")
    if case["mode"] == "all":
        t, k, p, q = [1.0] * m, [0] * m, [1.0] * m, [0.0] * m
    elif case["mode"] == "chat":
        t, k, p, q = [0.8] * m, [40] * m, [0.95] * m, [0.0] * m
    else:
        t = [rng.choice([0.0, 0.6, 0.8, 1.0, 1.3]) for _ in range(m)]
        k = [rng.choice([0, 0, 1, 20, 50, 1000]) for _ in range(m)]
        p = [rng.choice([1.0, 1.0, 0.8, 0.95, 0.5]) for _ in range(m)]
        q = [rng.choice([0.0, 0.0, 0.05, 0.1]) for _ in range(m)]
    s["temperature"], s["top_p"], s["min_p"] = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (t, p, q))
    s["top_k"] = _int32(k)
    s["tokens"] = torch.zeros(m, dtype=torch.int32, device="cuda")
    s["logp"] = torch.zeros(m, dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "plan":
        return _prepare_plan(case, s, gen)
    if op == "norm":
        return _prepare_norm(case, s, gen)
    if op == "sample":
        return _prepare_sample(case, s, gen, seed)
    t, h, d, p, lens, news = case["type"], case["heads"], case["d"], case["page"], _lens(case), _news(case)
    most = max(1, max(_up(n, p) for n in lens))
    s["count"] = len(lens) * most + 3
    order = torch.randperm(s["count"], generator=gen, device="cuda")[: len(lens) * most]
    s["pages"] = order.view(len(lens), most).to(torch.int32)
    s["lens"], s["q_starts"] = _int32(lens), _int32(_starts(news))
    # keys drift from page to page, a few of their channels are larger
    bump = 1 + 3 * (torch.rand(d, generator=gen, device="cuda") < 0.05)
    for name in ("k",) if op == "bounds" else ("k", "v"):
        cache = torch.empty(s["count"], h, p * _token_bytes(t, d), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (h * p * d))
        for at in range(0, s["count"], step):
            n = min(step, s["count"] - at)
            x = _normal(gen, n, h, p, d)
            codes, scales = _block_codes(t, (x + 0.7 * _normal(gen, n, h, 1, d)) * bump if name == "k" else x)
            cache[at : at + step, :, : p * _code_bytes(t, d)] = codes.flatten(2)
            cache[at : at + step, :, p * _code_bytes(t, d) :] = scales.view(torch.uint8).flatten(2)
        s[name + "_cache"] = cache
    s["bounds"] = torch.zeros(s["count"], h, _bound_bytes(d), dtype=torch.uint8, device="cuda")
    if op == "bounds":
        return s
    _plain_bounds(s | {"q_starts": _int32(_starts(lens))})       # as they stand after the new tokens are written
    new, hq = sum(news), h * case["group"]
    s["q"] = _normal(gen, new, hq, d).to(DTYPES[case["dtype"]])
    s["out"] = torch.zeros_like(s["q"])
    s["chosen"] = torch.full((new, h, case["budget"]), -1, dtype=torch.int32, device="cuda")
    rng = random.Random(seed)
    s["tree"] = None
    if case["tree"]:
        bits = [b for i, n in enumerate(news) for b in _ancestors(rng, n, i % 4 == 3)]
        s["tree"] = torch.tensor(bits, dtype=torch.int64, device="cuda")
    s["scale"] = 1 / math.sqrt(d)
    s["ws"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms: the plan
def _plain_plan(s):
    case, lens, news, pages, ring = s["case"], s["lens"].long(), s["news"].long(), s["pages"].long(), s["ring"].long()
    p, n, ld, count, rows = case["page"], s["lens"].shape[0], s["pages"].shape[1], s["ring"].shape[0], s["rows"]
    first, last = s["ring_at"][0], s["ring_at"][1]
    held, new = (lens + p - 1) // p, news.clamp(min=0)
    after = (lens + new + p - 1) // p
    need = torch.where(after <= ld, after - held, 0)
    upto = torch.cumsum(need, 0)
    fine = (after <= ld) & ((need == 0) | (upto <= last - first)) & (news >= 0)
    q_starts = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    # every row: its sequence, position and page
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(q_starts, row, right=True) - 1
    pos = lens[seq] + row - q_starts[seq]
    k = pos // p - held[seq]
    taken = ring[(first + (upto - need)[seq] + k.clamp(min=0)) % count]
    old = pages[seq, (pos // p).clamp(max=ld - 1)]
    page = torch.where(k >= 0, taken, old)
    ok = fine[seq]
    table = torch.nn.functional.pad(pages.flatten(), (0, 1))
    table[torch.where(ok, seq * ld + pos // p, n * ld)] = page
    # the pages of requests that are done go back
    done = news < 0
    back = torch.where(done, held, 0)
    j = torch.arange(ld, device="cuda")[None, :]
    to = (last + (torch.cumsum(back, 0) - back)[:, None] + j) % count
    ring = torch.nn.functional.pad(ring, (0, 1))
    ring[torch.where(done[:, None] & (j < held[:, None]), to, count)] = pages
    i32 = torch.int32
    return {"q_starts": q_starts.to(i32), "kv_lens": torch.where(fine, lens + new, 0).to(i32),
            "slots": torch.where(ok, page * p + pos % p, -1), "positions": torch.where(ok, pos, -1).to(i32),
            "next_lens": torch.where(done, 0, torch.where(fine, lens + new, lens)).to(i32), "pages": table[:-1].view(n, ld).to(i32),
            "ring": ring[:-1].to(i32), "next_at": torch.stack((first + torch.where(fine, need, 0).sum(), last + back.sum()))}


# ----------------------------------------------------------------------- plain forms: the cache
def _block_codes(t, x):
    """fp32 [..., D] -> (code bytes, fp16 scales [..., D/32]) by the GGML rule of the type (finite values)."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs()
    top = a.amax(-1, keepdim=True)
    if t == "q8_0":
        d = top / 127
    else:
        at = torch.where(a == top, torch.arange(32, device=x.device), 31).amin(-1, keepdim=True)
        d = torch.gather(b, -1, at) / -8
    v = b * torch.where(d != 0, 1 / d, 0.0)
    if t == "q8_0":
        codes = _round_away(v).to(torch.int8).view(torch.uint8).flatten(-2)
    else:
        q = torch.trunc((v + 8.5).clamp(0, 15)).to(torch.uint8)
        codes = (q[..., :16] | q[..., 16:] << 4).flatten(-2)
    return codes, d.to(torch.float16).squeeze(-1)


def _by127(x):
    """x / 127 to the nearest fp32 (torch multiplies by the reciprocal of a plain number)."""
    return x / torch.full((), 127.0, device=x.device)


def _power(e):
    """2^e in fp64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_away(v):
    """To the nearest whole number, halves away from zero, within [-127, 127]."""
    v = v.clamp(-127, 127)
    q = torch.trunc(v)
    return q + ((v - q).abs() >= 0.5) * torch.sign(v)


def _parts(cache, t, d, p):
    """Views of a cache's codes [pages][heads][P][bytes] and scales [pages][heads][P][D/32] (fp16)."""
    n = p * _code_bytes(t, d)
    return cache[..., :n].unflatten(-1, (p, -1)), cache[..., n:].view(torch.float16).unflatten(-1, (p, -1))


def _values(t, codes, scales):
    """fp32 values [..., D] of code bytes and their scales."""
    if t == "q8_0":
        v = codes.view(torch.int8).float().unflatten(-1, (-1, 32))
    else:
        c = codes.unflatten(-1, (-1, 16))
        v = torch.cat((c & 15, c >> 4), -1).float() - 8
    return (v * scales.float().unsqueeze(-1)).flatten(-2)


def _bound_parts(bounds, d):
    """Views of the bounds' codes int8 [pages][heads][2][D] and scales [pages][heads][D/32]."""
    return bounds[..., : 2 * d].view(torch.int8).unflatten(-1, (2, d)), bounds[..., 2 * d : 2 * d + d // 32 * 2].view(torch.float16)


def _bound_values(s):
    codes, scales = _bound_parts(s["bounds"], s["case"]["d"])
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[:, :, None, :, None]).flatten(-2)


def _up_half(x):
    """x >= 0 rounded up to fp16."""
    h = x.to(torch.float16)
    return (h.view(torch.int16) + (h.float() < x)).to(torch.int16).view(torch.float16)


def _plain_bounds(s):
    case = s["case"]
    t, d, p = case["type"], case["d"], case["page"]
    lens = s["lens"].long()
    news = (s["q_starts"][1:] - s["q_starts"][:-1]).long()
    k0, k1 = (lens - news) // p, torch.where(news > 0, (lens - 1) // p + 1, 0)
    k = torch.arange(s["pages"].shape[1], device="cuda")[None, :]
    seq, k = torch.nonzero((k >= k0[:, None]) & (k < k1[:, None]), as_tuple=True)
    page = s["pages"][seq, k].long()
    codes, scales = _parts(s["k_cache"], t, d, p)
    v = _values(t, codes[page], scales[page])                                             # [pages, H, P, D]
    have = (k[:, None] * p + torch.arange(p, device="cuda") < lens[seq][:, None])[:, None, :, None]
    lo, hi = torch.where(have, v, math.inf).amin(2), torch.where(have, v, -math.inf).amax(2)
    b = torch.stack((lo, hi), 2).unflatten(-1, (-1, 32))                                 # [pages, H, 2, D/32, 32]
    half = _up_half(_by127(b.abs().amax((2, 4))))
    u = b / torch.where(half > 0, half.float(), 1.0)[:, :, None, :, None]
    q = torch.cat((torch.floor(u[:, :, :1]), torch.ceil(u[:, :, 1:])), 2).clamp(-127, 127).flatten(-2)
    bc, bs = _bound_parts(s["bounds"], d)
    bc[page], bs[page] = q.to(torch.int8), half


def _plain_chosen(s):
    """For each new token and key/value head the numbers of its pages, ascending, then -1."""
    case = s["case"]
    d, p, h, g = case["d"], case["page"], case["heads"], case["group"]
    lens, first = s["lens"].long(), s["q_starts"][:-1].long()
    news = s["q_starts"][1:].long() - first
    n, most = max(1, case["new"]), s["pages"].shape[1]
    i = torch.arange(n, device="cuda")
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)                            # [S, n]
    x = s["q"][row].float().unflatten(2, (h, g)).unflatten(-1, (-1, 32))                  # [S, n, H, G, b, 32]
    dq = _by127(x.abs().amax(-1, keepdim=True))
    a = _round_away(x * torch.where(dq != 0, 1 / dq, 0.0)).permute(0, 2, 4, 1, 3, 5).flatten(3, 4)   # [S, H, b, nG, 32]
    codes, scales = _bound_parts(s["bounds"], d)
    page = s["pages"].long()
    c = codes[page].float().unflatten(-1, (-1, 32)).permute(0, 2, 4, 3, 5, 1)            # [S, H, b, 2, 32, pages]
    dots = torch.matmul(a.clamp(max=0), c[..., 0, :, :]) + torch.matmul(a.clamp(min=0), c[..., 1, :, :])   # whole numbers
    db = scales[page].float().permute(0, 2, 3, 1)[:, :, :, None, :]                      # [S, H, b, 1, pages]
    terms = (dq.squeeze(-1).permute(0, 2, 4, 1, 3).flatten(3, 4).unsqueeze(-1) * db) * dots
    score = functools.reduce(torch.add, terms.unbind(2), torch.zeros((), device="cuda"))           # block after block, in fp32
    score = score.unflatten(2, (n, g)).amax(3).permute(0, 2, 1, 3).double()               # [S, n, H, pages]
    k = torch.arange(most, device="cuda")
    at = (lens - news)[:, None] + i[None, :]                                              # the token's place
    seen = torch.where(i[None, :] < news[:, None], (at if s["tree"] is None else (lens - 1)[:, None].expand_as(at)) // p, -1)
    old = (at if s["tree"] is None else (lens - news)[:, None].expand_as(at)) // p - (case["recent"] - 1)
    must = (k < case["sinks"]) | (k >= old[:, :, None])
    score = torch.where(must[:, :, None], math.inf, score)
    score = torch.where((k <= seen[:, :, None])[:, :, None], score, -math.inf)
    score, order = torch.sort(score, dim=-1, descending=True, stable=True)
    top = torch.nn.functional.pad(torch.where(score[..., : case["budget"]] > -math.inf, order[..., : case["budget"]], most), (0, max(0, case["budget"] - most)), value=most)
    top = top.sort(-1).values
    return torch.where(top < most, top, -1)[i[None, :] < news[:, None]].to(torch.int32)


def _plain_sparse(s):
    case = s["case"]
    t, d, p, h, g = case["type"], case["d"], case["page"], case["heads"], case["group"]
    chosen = _plain_chosen(s)
    lens, first = s["lens"].long(), s["q_starts"][:-1].long()
    news = s["q_starts"][1:].long() - first
    tok = torch.arange(chosen.shape[0], device="cuda")
    seq = torch.searchsorted(s["q_starts"], tok, right=True) - 1
    page = s["pages"][seq[:, None, None], chosen.clamp(min=0).long()].long()              # [T, H, B]
    head = torch.arange(h, device="cuda")[None, :, None]

    def gather(name):
        codes, scales = _parts(s[name], t, d, p)
        return _values(t, codes[page, head], scales[page, head]).flatten(2, 3)            # [T, H, B * P, D]

    pos = (chosen[..., None].long() * p + torch.arange(p, device="cuda")).flatten(2)
    nb = pos - (lens - news)[seq][:, None, None]                                          # place among the new tokens
    i = (tok - first[seq])[:, None, None]
    seen = nb <= i if s["tree"] is None else (nb < 0) | (nb < 64) & ((s["tree"][:, None, None] >> nb.clamp(0, 63)) & 1 == 1)
    seen = seen & (pos < lens[seq][:, None, None]) & (chosen >= 0).repeat_interleave(p, -1)
    q = s["q"].float().unflatten(1, (h, g))
    sc = (torch.matmul(q, gather("k_cache").transpose(2, 3)) * s["scale"]).masked_fill(~seen[:, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(e, gather("v_cache")) / total, 0.0)
    return {"chosen": chosen, "out": o.flatten(1, 2).to(s["q"].dtype)}


# ------------------------------------------------------------- plain forms: norms and sampling
def _mx4_values(x):
    """fp32 rows at their MX4 values: the scale is 2^(floor(log2 max|x|) - 2), the codes are rounded to the nearest E2M1
    value, ties to the even code, beyond 6 to 6."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    unit = _power((torch.frexp(top)[1] - 3).clamp(min=-127)).float()
    a = torch.where(top > 0, b.abs() / unit, 0.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return ((torch.round(a / step) * step).clamp(max=6.0) * torch.sign(b) * unit).flatten(-2)


def _q8_values(x):
    b = x.unflatten(-1, (-1, 32))
    d = _by127(b.abs().amax(-1, keepdim=True))
    return (_round_away(b * torch.where(d != 0, 1 / d, 0.0)) * d.to(torch.float16).float()).flatten(-2)


def _rms(x, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _plain_norm(s):
    x, form = s["x"].float(), s["case"]["form"]
    if s["w_post"] is not None:
        x = _rms(x, s["eps"]) * s["w_post"]
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = (s["h"].float() + s["scale"] * x).to(s["h"].dtype)
    y = _rms(h.float(), s["eps"]) * s["w_pre"]
    if form in ("q8", "mx4"):
        return {"h": h, "y": (_q8_values(y) if form == "q8" else _mx4_values(y)).to(torch.bfloat16)}
    return {"h": h, "y": y.to(DTYPES[form])}


def _plain_sample(s):
    z = s["logits"].double()
    m, v = z.shape
    t, k = s["temperature"].double()[:, None], s["top_k"].long()[:, None]
    p, q = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = torch.exp((z - z[:, :1]) / torch.where(t > 0, t, 1.0))
    rank = torch.arange(v, device="cuda")[None, :]
    keep = rank < torch.where((k <= 0) | (k > v), v, k)
    w = torch.where(keep, w, 0.0)
    upto = torch.cumsum(w, -1)
    keep &= (rank == 0) | (upto - w < p * upto[:, -1:]) | (p >= 1)
    keep &= (w >= q) | (rank == 0)
    keep &= (rank == 0) | (t > 0)
    w = torch.where(keep, w, 0.0)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    upto = torch.cumsum(kept, -1)
    total = upto[:, -1:]
    tokens = (upto > s["u"].double()[:, None] * total).to(torch.int8).argmax(-1)
    logp = torch.log(kept.gather(1, tokens[:, None]) / total).squeeze(1)
    return {"tokens": tokens.to(torch.int32), "logp": logp.float()}


def _own(s):
    import block_quantized_matmul_gb300 as qmm

    case = s["case"]
    op = case["op"]
    if op == "plan":
        n, ld = s["pages"].shape
        qmm.qmm_cache_plan(s["lens"], s["news"], n, case["page"], s["pages"], ld, s["ring"], s["ring"].numel(), s["ring_at"], s["rows"],
                           s["q_starts"], s["kv_lens"], s["slots"], s["positions"], s["next_lens"], s["next_at"])
        return {x: s[x] for x in ("q_starts", "kv_lens", "slots", "positions", "next_lens", "pages", "ring", "next_at")}
    if op == "norm":
        m, n, form = case["rows"], case["n"], case["form"]
        ldg = n if case["gate"] == "rows" else 0
        args = (case["x"], s["x"], n, case["h"], s["h"], n, m, n, s["w_post"], s["gate"], ldg, s["scale"], s["w_pre"], s["eps"], s["h_out"], n)
        if form == "q8":
            qmm.qmm_norm_q8(*args, s["a_q"], s["a_d"])
            y = (s["a_q"].view(m, -1, 32).float() * s["a_d"].float().unsqueeze(-1)).view(m, n).to(torch.bfloat16)
            return {"h": s["h_out"], "y": y}
        if form == "mx4":
            qmm.qmm_norm_mx4(*args, s["codes"], s["scales"])
            qmm.qmm_mx4_dequantize(s["codes"], s["scales"], m, n, "bf16", s["y"], n)
        else:
            qmm.qmm_norm(*args, form, s["y"], n)
        return {"h": s["h_out"], "y": s["y"]}
    if op == "sample":
        v = case["v"]
        qmm.qmm_sample(case["dtype"], s["logits"], v, case["rows"], v, s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["tokens"], s["logp"])
        return {"tokens": s["tokens"], "logp": s["logp"]}
    t, h, d, p, n = case["type"], case["heads"], case["d"], case["page"], s["count"]
    table, ld, seqs = s["pages"], s["pages"].shape[1], case["seqs"]
    if op == "bounds":
        qmm.qmm_cache_bounds(t, s["k_cache"], n, p, h, d, table, ld, s["q_starts"], s["lens"], seqs, sum(_news(case)), case["new"], s["bounds"])
        return {"bounds": _bound_values(s)}
    hq, new, b = h * case["group"], s["q"].shape[0], case["budget"]
    qmm.qmm_cache_select(s["bounds"], n, p, h, d, table, ld, s["q_starts"], s["lens"], seqs, case["dtype"], s["q"], hq * d, new, hq, s["tree"],
                         case["new"], case["hi"], case["sinks"], case["recent"], b, s["chosen"], s["ws"], WORKSPACE)
    qmm.qmm_cache_attend_chosen(t, s["k_cache"], s["v_cache"], n, p, h, d, table, ld, s["q_starts"], s["lens"], seqs, case["dtype"], s["q"], hq * d, new, hq,
                                s["tree"], s["scale"], s["chosen"], b, s["out"], hq * d, None, s["ws"], WORKSPACE)
    return {"chosen": s["chosen"], "out": s["out"]}


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "bounds":
        _plain_bounds(s)
        return {"bounds": _bound_values(s)}
    return {"plan": _plain_plan, "sparse": _plain_sparse, "norm": _plain_norm, "sample": _plain_sample}[op](s)


# ---------------------------------------------------------------------------------- exact, in fp64
def _exact_plan(s):
    case, p = s["case"], s["case"]["page"]
    lens, news, pages, ring = (s[x].tolist() for x in ("lens", "news", "pages", "ring"))
    (first, last), count, ld = s["ring_at"].tolist(), len(ring), s["pages"].shape[1]
    free, line, starts, kv, nxt, slots, places = last - first, 0, [0], [], [], [], []
    taken, back = 0, 0
    new_ring = list(ring)
    for s_, (n, new) in enumerate(zip(lens, news)):
        held = _up(n, p)
        if new < 0:
            for page in pages[s_][:held]:
                new_ring[(last + back) % count] = page
                back += 1
            kv.append(0)
            nxt.append(0)
            starts.append(starts[-1])
            continue
        need = _up(n + new, p) - held
        fits = held + need <= ld
        line += need if fits else 0
        if fits and (need == 0 or line <= free):
            for j in range(need):
                pages[s_][held + j] = ring[(first + taken) % count]
                taken += 1
            slots += [pages[s_][(n + i) // p] * p + (n + i) % p for i in range(new)]
            places += range(n, n + new)
            kv.append(n + new)
            nxt.append(n + new)
        else:
            slots += [-1] * new
            places += [-1] * new
            kv.append(0)
            nxt.append(n)
        starts.append(starts[-1] + new)
    return {"q_starts": _int32(starts), "kv_lens": _int32(kv), "slots": torch.tensor(slots, dtype=torch.int64, device="cuda"), "positions": _int32(places),
            "next_lens": _int32(nxt), "pages": _int32(pages), "ring": _int32(new_ring), "next_at": torch.tensor([first + taken, last + back], device="cuda")}


def _exact_tokens(cache, t, h, d, p, page, off):
    """fp64 [tokens][D] of one head from the bytes of a cache."""
    n, cb = d // 32, _code_bytes(t, d)
    base = (page * cache.shape[1] + h) * (p * _token_bytes(t, d))
    flat = cache.reshape(-1)
    e = torch.arange(d, device="cuda")
    at = (base + off * cb)[:, None]
    if t == "q8_0":
        q = flat[at + e].double()
        q = torch.where(q > 127, q - 256, q)
    else:
        byte = flat[at + e // 32 * 16 + e % 16]
        q = torch.where(e % 32 < 16, byte % 16, byte // 16).double() - 8
    half = (base + p * cb + off * 2 * n)[:, None] + 2 * torch.arange(n, device="cuda")
    return q * torch.stack((flat[half], flat[half + 1]), -1).view(torch.float16).squeeze(-1).double().repeat_interleave(32, -1)


def _exact_bounds(s):
    case = s["case"]
    t, h, d, p = case["type"], case["heads"], case["d"], case["page"]
    out = _bound_values(s).double()
    touched = _touched(case)
    table = s["pages"].long()
    pages = torch.stack([table[a, k] for a, k, _ in touched]) if touched else table.new_zeros(0)
    counts = torch.tensor([n for _, _, n in touched], device="cuda")
    off = torch.arange(p, device="cuda")
    for head in range(h):
        v = _exact_tokens(s["k_cache"], t, head, d, p, pages.repeat_interleave(p), off.repeat(len(touched))).view(-1, p, d)
        gone = (off >= counts[:, None])[..., None]
        lo, hi = v.masked_fill(gone, 1e30).min(1).values, v.masked_fill(gone, -1e30).max(1).values
        for b in range(d // 32):
            at = slice(32 * b, 32 * b + 32)
            top = torch.maximum(lo[:, at].abs().max(1).values, hi[:, at].abs().max(1).values) / 127
            # the least multiple of fp16's spacing that is not below
            unit = _power((torch.frexp(top)[1] - 11).clamp(min=-24))
            scale = (torch.ceil(top.float().double() / unit) * unit)[:, None]
            one = torch.where(scale > 0, scale, 1.0)
            out[pages, head, 0, at] = torch.floor((lo[:, at] / one).float()).clamp(-127, 127).double() * scale
            out[pages, head, 1, at] = torch.ceil((hi[:, at] / one).float()).clamp(-127, 127).double() * scale
    return {"bounds": out}


def _exact_sparse(s):
    case = s["case"]
    t, h, d, p, g = case["type"], case["heads"], case["d"], case["page"], case["group"]
    lens, news, table = _lens(case), _news(case), s["pages"].long()
    flat = s["bounds"].view(torch.int8)
    halves = s["bounds"][..., 2 * d : 2 * d + d // 32 * 2].contiguous().view(torch.float16).float()
    chosen, outs, at = [], [], 0
    off = torch.arange(p, device="cuda")
    if sum(news) * h * g * d > 1 << 19:
        return None
    for i, (n, new) in enumerate(zip(lens, news)):
        if new == 0:
            continue
        first = n - new
        for r in range(new):
            last = n - 1 if case["tree"] else first + r
            pages = last // p + 1
            ids = table[i, :pages]
            must = set(range(min(case["sinks"], pages))) | set(range(max(0, (first if case["tree"] else last) // p - case["recent"] + 1), pages))
            for head in range(h):
                best = torch.full((pages,), -math.inf, device="cuda")
                lo, hi = flat[ids, head, :d].double(), flat[ids, head, d : 2 * d].double()
                for x in s["q"][at + r, head * g : head * g + g].float():
                    score = torch.zeros(pages, device="cuda")
                    for b in range(d // 32):
                        w = slice(32 * b, 32 * b + 32)
                        dq = x[w].abs().max().double().div(127).float()
                        v = x[w] * (1 / dq if dq > 0 else torch.zeros_like(dq))
                        a = (torch.floor(v.abs().double() + 0.5) * torch.sign(v)).clamp(-127, 127)
                        dot = torch.where(a > 0, hi[:, w] * a, lo[:, w] * a).sum(1).float()
                        score = score + (dq * halves[ids, head, b]) * dot
                    best = torch.maximum(best, score)
                ranks = sorted(range(pages), key=lambda j, v=best.tolist(): (j not in must, 0.0 if j in must else -v[j], j))
                pick = sorted(ranks[: case["budget"]])
                chosen.append(pick + [-1] * (case["budget"] - len(pick)))
                pick = torch.tensor(pick, device="cuda")
                pos = (pick[:, None] * p + off).flatten()
                page = table[i, pick].repeat_interleave(p)
                if case["tree"]:
                    bits = int(s["tree"][at + r])
                    allow = torch.tensor([bits >> j & 1 for j in range(new)], device="cuda", dtype=torch.bool)
                    seen = (pos < first) | (pos < n) & allow[(pos - first).clamp(0, new - 1)]
                else:
                    seen = pos <= last
                k, v = (_exact_tokens(s[name], t, head, d, p, page[seen], (pos % p)[seen]) for name in ("k_cache", "v_cache"))
                q = s["q"][at + r, head * g : head * g + g].double()
                outs.append(torch.softmax(q @ k.t() * s["scale"], -1) @ v)
        at += new
    if not outs:
        return None
    return {"chosen": _int32(chosen).view(-1, h, case["budget"]), "out": torch.stack(outs).view(-1, h * g, d)}


def _exact_norm(s):
    case = s["case"]
    n = case["n"]
    x = s["x"].double()
    if case["post"]:
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / n + s["eps"]) * s["w_post"].double()
    if s["gate"] is not None:
        x = s["gate"].double() * x
    h = s["h"].double() + s["scale"] * x
    r = h.to(s["h"].dtype).double()                      # the stream as it is stored
    y = r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / n + s["eps"]) * s["w_pre"].double()
    if case["form"] in ("q8", "mx4"):
        b = y.reshape(-1, 32)
        top = b.abs().max(1, keepdim=True).values
        if case["form"] == "q8":
            unit = top / 127
            y = torch.floor((b / torch.where(unit > 0, unit, 1.0)).abs() + 0.5) * torch.sign(b) * unit.to(torch.float16).double()
        else:
            unit = _power((torch.frexp(top)[1] - 3).clamp(min=-127))
            grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
            # the borders between neighbours; one that is met goes to the even code
            mid = (grid[1:] + grid[:-1]) / 2
            u = b.abs() / unit
            code = torch.where(torch.bucketize(u, mid) % 2 == 0, torch.bucketize(u, mid), torch.bucketize(u, mid, right=True))
            y = grid[code] * torch.sign(b) * unit
        y = y.view(h.shape)
    return {"h": h, "y": y}


def _exact_sample(s):
    tokens, logps = [], []
    for i in range(s["case"]["rows"]):
        z = s["logits"][i].double()
        t, k, p, q, u = (float(s[x][i]) for x in ("temperature", "top_k", "top_p", "min_p", "u"))
        best = int(torch.nonzero(z == z.max())[0])
        if t <= 0:
            tokens.append(best)
            logps.append(0.0)
            continue
        w = torch.exp((z - z[best]) / t)
        order = torch.argsort(-z, stable=True)
        if 0 < k < len(z):
            order = order[: int(k)]
        if p < 1:
            mass = w[order]
            before = torch.cumsum(mass, 0) - mass
            order = order[: max(1, int((before < p * mass.sum()).sum()))]
        if q > 0:
            order = order[: max(1, int((w[order] >= q).sum()))]
        index = torch.sort(order).values
        upto = torch.cumsum(w[index], 0)
        at = min(int((upto <= u * upto[-1]).sum()), len(index) - 1)
        tokens.append(int(index[at]))
        logps.append(float(torch.log(w[index[at]] / upto[-1])))
    return {"tokens": _int32(tokens), "logp": torch.tensor(logps, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "bounds": _exact_bounds, "sparse": _exact_sparse, "norm": _exact_norm, "sample": _exact_sample}[case["op"]](s)
