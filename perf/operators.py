"""The operators of a block-quantized decoder step beyond the tiled products, as cases to be measured.

  quantize  rows -> microscaled 4-bit floating point (MX4: E2M1 codes, one E8M0 scale per 32) and back to values
  linear    rows quantized to MX4 times an MX4 weight
  cache     the keys and values of new tokens quantized as they are written into a paged cache, and the
            sequences read back from it
  attend    attention of a sequence's new tokens (one token, or a tree of drafted tokens) over that cache

With `own` false, run() computes each in elementary torch operations in fp32; with `own` true it makes the
library's calls.  exact() computes them in fp64.

Layouts (both sides read and write the same buffers):
  MX4 operand of R rows of K (K % 32 == 0): codes uint8 [R][K/2], element 2i in the low nibble of byte i;
    scales in blocks of 512 bytes for 128 rows x 4 blocks of 32, block (R/128, K/128), byte
    16*(r % 32) + 4*((r % 128)/32) + (b % 4); blocks past the last row or column hold 0.
  Cache page of P tokens: for each head [P][D] codes (q8_0: int8; q4_0: [P][D/2] bytes, byte j of a block of 32
    holds element j low and j + 16 high), then [P][D/32] fp16 scales.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
WORKSPACE = 64 << 20   # bytes a server keeps for the attention's partial results


def listed():
    return [
        # the activations of one decode step of eight sequences
        {"name": "quantize decode rows", "op": "quantize", "rows": 8, "k": 4096, "dtype": "bf16"},
        # a weight matrix at load time
        {"name": "quantize weight", "op": "quantize", "rows": 14336, "k": 4096, "dtype": "f32"},
        # one token through the up projection of a feed-forward block
        {"name": "linear one token", "op": "linear", "m": 1, "k": 4096, "n": 14336, "dtype": "bf16", "out": "bf16"},
        # a ragged batch of tokens, a width that is no multiple of any tile, fp32 results
        {"name": "linear ragged", "op": "linear", "m": 37, "k": 4128, "n": 4099, "dtype": "f32", "out": "f32"},
        # a short prompt through the up projection
        {"name": "linear prompt", "op": "linear", "m": 512, "k": 4096, "n": 14336, "dtype": "bf16", "out": "bf16"},
        # a long prompt through the down projection
        {"name": "linear long prompt", "op": "linear", "m": 8192, "k": 14336, "n": 4096, "dtype": "bf16", "out": "bf16"},
        # a decode step of a batch of short sequences: one token each is written, the sequences are read back
        {"name": "cache decode step", "op": "cache", "type": "q8_0", "seqs": 16, "lo": 1, "hi": 60, "new": 1, "heads": 8, "d": 128, "page": 16, "dtype": "bf16"},
        # four prompts are written as a whole and read back (for an attention over dense keys and values)
        {"name": "cache prompts", "op": "cache", "type": "q4_0", "seqs": 4, "lo": 3000, "hi": 16384, "new": 16384, "heads": 8, "d": 128, "page": 64, "dtype": "f16"},
        # one token of one short sequence: latency
        {"name": "attend one token", "op": "attend", "type": "q8_0", "seqs": 1, "lo": 777, "hi": 777, "new": 1, "tree": False, "heads": 8, "group": 4, "d": 128, "page": 16, "dtype": "bf16"},
        # a batch of decode steps at ragged lengths, one of them empty
        {"name": "attend batch", "op": "attend", "type": "q8_0", "seqs": 64, "lo": 0, "hi": 8192, "new": 1, "tree": False, "heads": 8, "group": 4, "d": 128, "page": 64, "dtype": "bf16"},
        # trees of drafted tokens of eight sequences, checked against the target model in one step
        {"name": "attend trees", "op": "attend", "type": "q4_0", "seqs": 8, "lo": 200, "hi": 4096, "new": 32, "tree": True, "heads": 8, "group": 4, "d": 128, "page": 64, "dtype": "f16"},
        # one token over a very long sequence: the work of a few heads has to be split over its length
        {"name": "attend long", "op": "attend", "type": "q8_0", "seqs": 1, "lo": 500001, "hi": 500001, "new": 1, "tree": False, "heads": 4, "group": 8, "d": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "cache", "attend", "attend"])
    if op == "quantize":
        k = 32 * _log(rng, 4, 448)
        return {"op": op, "rows": _log(rng, 8, min(14336, (1 << 25) // k)), "k": k, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op == "linear":
        k, n = 32 * _log(rng, 16, 448), _log(rng, 500, 16384)
        m = _log(rng, 1, min(8192, (1 << 38) // (k * n)))
        # fp32 results are asked for where logits are: rows of moderate length
        return {"op": op, "m": m, "k": k, "n": n, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "out": rng.choice(["f16", "bf16", "f32" if k <= 4128 else "bf16"])}
    c = {"op": op, "type": rng.choice(["q8_0", "q4_0"]), "seqs": _log(rng, 1, 48), "heads": rng.choice([1, 2, 4, 8]),
         "d": rng.choice([64, 96, 128, 256]), "page": rng.choice([16, 32, 64, 128, 256])}
    most = min(65536, (1 << 27) // (c["seqs"] * c["heads"] * c["d"]))
    if op == "attend":
        tree = rng.random() < 0.4
        c |= {"new": rng.randrange(2, 65) if tree else rng.choice([1, 1, rng.randrange(2, 17)]), "tree": tree,
              "group": rng.choice([1, 2, 3, 4, 7, 8, 16]), "dtype": rng.choice(["f16", "bf16"])}
        most = min(most, (1 << 28) // (c["seqs"] * c["heads"] * c["group"] * c["new"]))
    c["hi"] = _log(rng, 20, max(20, most))
    c["lo"] = rng.randrange(0, c["hi"] + 1)
    if op == "cache":
        c |= {"new": rng.choice([1, _log(rng, 1, c["hi"])]), "dtype": rng.choice(["f32", "f16", "bf16"])}
    return c


# ------------------------------------------------------------------------------------------- sizes
def _lens(case):
    """The sequences' lengths: spread from lo to hi, in a fixed odd order."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * ((i * 7919 + n // 2) % n) // (n - 1) for i in range(n)]


def _news(case):
    return [min(n, case["new"]) for n in _lens(case)]


def _code_bytes(t, d):
    return d if t == "q8_0" else d // 2


def _token_bytes(t, d):
    return _code_bytes(t, d) + d // 32 * 2


def _mx4_bytes(rows, k):
    return rows * (k // 2 + k // 32)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["k"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * _mx4_bytes(case["rows"], case["k"]), "flops": 4 * n}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": m * k * SIZE[case["dtype"]] + _mx4_bytes(n, k) + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    t, h, d = case["type"], case["heads"], case["d"]
    lens, news = sum(_lens(case)), sum(_news(case))
    if op == "cache":
        s = SIZE[case["dtype"]] * d
        return {"bytes": 2 * h * ((news + lens) * s + (news + lens) * _token_bytes(t, d)), "flops": 2 * h * d * (4 * news + lens)}
    rows = sum(a * b for a, b in zip(_lens(case), _news(case))) * h * case["group"]
    return {"bytes": 2 * h * lens * _token_bytes(t, d) + 2 * news * h * case["group"] * d * SIZE[case["dtype"]], "flops": 4 * rows * d}


# ------------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, k):
    """Rows of a layer's input: normal values, a few channels twenty times larger."""
    x = _normal(gen, rows, k)
    big = torch.rand(k, generator=gen, device="cuda") < 0.01
    return torch.where(big, 20 * x, x)


def _pages(case, gen):
    """The page table: the sequences' pages lie scattered over the pool, a few pages of which are free."""
    lens, p = _lens(case), case["page"]
    most = max(1, max((n + p - 1) // p for n in lens))
    count = len(lens) * most + 3
    order = torch.randperm(count, generator=gen, device="cuda")[: len(lens) * most]
    return order.view(len(lens), most).to(torch.int32), count


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "quantize":
        r, k = case["rows"], case["k"]
        s["x"] = _activations(gen, r, k).to(DTYPES[case["dtype"]])
        s["codes"] = torch.zeros(r, k // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(-(-r // 128) * -(-k // 128) * 512, dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros_like(s["x"])
        return s
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["w_codes"], s["w_scales"] = _mx4_pack(*_mx4_codes(0.02 * _normal(gen, n, k)))
        s["x"] = _activations(gen, m, k).to(DTYPES[case["dtype"]])
        s["y"] = torch.zeros(m, n, dtype=DTYPES[case["out"]], device="cuda")
        s["ws"] = torch.zeros(-(-(m * k // 2) // 256) * 256 + -(-m // 128) * -(-k // 128) * 512, dtype=torch.uint8, device="cuda")
        return s
    t, h, d, p, lens, news = case["type"], case["heads"], case["d"], case["page"], _lens(case), _news(case)
    s["pages"], s["count"] = _pages(case, gen)
    s["lens"], s["starts"], s["q_starts"] = _int32(lens), _int32(_starts(lens)), _int32(_starts(news))
    # what the cache already holds: normal keys and values, a few key channels larger, all pages filled
    bump = 1 + 3 * (torch.rand(d, generator=gen, device="cuda") < 0.05)
    for name in ("k", "v"):
        cache = torch.empty(s["count"], h, p * _token_bytes(t, d), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (h * p * d))
        for at in range(0, s["count"], step):
            x = _normal(gen, min(step, s["count"] - at), h, p, d)
            codes, scales = _block_codes(t, x * bump if name == "k" else x)
            cache[at : at + step, :, : p * _code_bytes(t, d)] = codes.flatten(2)
            cache[at : at + step, :, p * _code_bytes(t, d) :] = scales.view(torch.uint8).flatten(2)
        s[name + "_cache"] = cache
    total, new = sum(lens), sum(news)
    if op == "cache":
        dt = DTYPES[case["dtype"]]
        s["k"], s["v"] = (_normal(gen, new, h, d).to(dt) for _ in range(2))
        seq = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news)).cuda()
        pos = (s["lens"][seq] - s["q_starts"][1:][seq] + torch.arange(new, device="cuda")).long()
        s["slots"] = s["pages"][seq, pos // p].long() * p + pos % p
        s["k_out"], s["v_out"] = (torch.zeros(total, h, d, dtype=dt, device="cuda") for _ in range(2))
        return s
    s["q"] = _normal(gen, new, h * case["group"], d).to(DTYPES[case["dtype"]])
    s["out"] = torch.zeros_like(s["q"])
    rng = random.Random(seed)
    s["tree"] = None
    if case["tree"]:
        bits = [b for i, n in enumerate(news) for b in _ancestors(rng, n, i % 4 == 3)]
        s["tree"] = torch.tensor(bits, dtype=torch.int64, device="cuda")
    s["scale"] = 1 / math.sqrt(d)
    s["ws"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------- plain forms
def _mx4_codes(x):
    """fp32 rows -> (codes [R][K] 0..15, E8M0 scales [R][K/32]): the scale is 2^(floor(log2 max|x|) - 2), the codes
    are rounded to the nearest E2M1 value, ties to the even code, beyond 6 to 6; a block that holds an infinity or a
    NaN has scale 255."""
    r, k = x.shape
    b = x.view(r, k // 32, 32)
    top = b.abs().amax(-1)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine, top, 0.0))[1] + (127 - 3)
    e = torch.where(top > 0, e.clamp(0, 254), 0)
    v = b * ((254 - e) << 23).to(torch.int32).view(torch.float32).unsqueeze(-1)
    a = v.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    c = torch.where(fine.unsqueeze(-1), c + 8 * torch.signbit(v), 0)
    return c.view(r, k).to(torch.uint8), torch.where(fine, e, 255).to(torch.uint8)


def _mx4_pack(codes, scales):
    """Codes and scales as the operand's two buffers."""
    r, kb = scales.shape
    r128, k4 = -(-r // 128), -(-kb // 4)
    s = torch.nn.functional.pad(scales, (0, 4 * k4 - kb, 0, 128 * r128 - r))
    s = s.view(r128, 4, 32, k4, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return codes[:, 0::2] | codes[:, 1::2] << 4, s


def _mx4_values(codes, scales):
    """The operand's values in fp32."""
    r, k = codes.shape[0], 2 * codes.shape[1]
    r128, k4 = -(-r // 128), -(-k // 128)
    e = scales.view(r128, k4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * r128, 4 * k4)[:r, : k // 32].to(torch.int32)
    s = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)
    s = torch.where(e < 255, s, float("nan"))
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).int()].view(r, k // 32, 32)
    return (v * s.unsqueeze(-1)).view(r, k)


def _block_codes(t, x):
    """fp32 [..., D] -> (code bytes, fp16 scales [..., D/32]) by the GGML rule of the type; a block with no finite
    fp16 scale has scale NaN and codes 0."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs()
    top = a.amax(-1, keepdim=True)
    if t == "q8_0":
        d = top / 127
    else:
        at = torch.where(a == top, torch.arange(32, device=x.device), 31).amin(-1, keepdim=True)
        d = torch.gather(b, -1, at) / -8
    half = d.to(torch.float16)
    fine = torch.isfinite(half)
    v = b * torch.where(d != 0, 1 / d, 0.0)
    if t == "q8_0":
        v = torch.nan_to_num(v, nan=0.0, posinf=127.0, neginf=-127.0).clamp(-127, 127)
        q = torch.trunc(v)
        q = q + ((v - q).abs() >= 0.5) * torch.sign(v)
        codes = torch.where(fine, q, 0).to(torch.int8).view(torch.uint8).flatten(-2)
    else:
        v = torch.nan_to_num(v + 8.5, nan=0.0, posinf=15.0, neginf=0.0).clamp(0, 15)
        q = torch.where(fine, torch.trunc(v), 0).to(torch.uint8)
        codes = (q[..., :16] | q[..., 16:] << 4).flatten(-2)
    return codes, torch.where(fine, half, float("nan")).squeeze(-1)


def _parts(cache, t, d, p):
    """Views of a cache's codes [pages][heads][P][bytes] and scales [pages][heads][P][D/32] (fp16)."""
    n = p * _code_bytes(t, d)
    return cache[..., :n].unflatten(-1, (p, -1)), cache[..., n:].view(torch.float16).unflatten(-1, (p, -1))


def _gather(cache, t, d, p, page, off):
    """fp32 values [..., heads, D] of the tokens at (page, off)."""
    codes, scales = _parts(cache, t, d, p)
    c, s = codes[page, :, off], scales[page, :, off].float()
    if t == "q8_0":
        v = c.view(torch.int8).float().unflatten(-1, (-1, 32))
    else:
        c = c.unflatten(-1, (-1, 16))
        v = torch.cat((c & 15, c >> 4), -1).float() - 8
    return (v * s.unsqueeze(-1)).flatten(-2)


def _plain_cache(s):
    case = s["case"]
    t, d, p = case["type"], case["d"], case["page"]
    for name in ("k", "v"):
        codes, scales = _parts(s[name + "_cache"], t, d, p)
        c, f = _block_codes(t, s[name].float())
        at = (s["slots"] // p, slice(None), s["slots"] % p)
        codes[at], scales[at] = c, f
    n = s["k_out"].shape[0]
    tok = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["starts"], tok, right=True) - 1
    pos = tok - s["starts"][seq]
    page = s["pages"][seq, pos // p].long()
    dt = s["k"].dtype
    return {"k": _gather(s["k_cache"], t, d, p, page, pos % p).to(dt), "v": _gather(s["v_cache"], t, d, p, page, pos % p).to(dt)}


def _plain_attend(s):
    case = s["case"]
    t, d, p, h, g = case["type"], case["d"], case["page"], case["heads"], case["group"]
    lens = s["lens"].long()
    first = s["q_starts"][:-1].long()
    news = s["q_starts"][1:].long() - first
    most, n = max(1, case["hi"]), max(1, case["new"])
    pos = torch.arange(most, device="cuda")
    page = s["pages"][:, (pos // p).clamp(max=s["pages"].shape[1] - 1)].long()
    off = (pos % p).expand_as(page)
    k, v = (_gather(s[name + "_cache"], t, d, p, page, off) for name in ("k", "v"))     # [S, L, H, D]
    i = torch.arange(n, device="cuda")
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)                           # [S, n]
    q = s["q"][row].float().unflatten(2, (h, g))                                        # [S, n, H, G, D]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                                          # [S, H, G*n, D]
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                            # [S, H, G*n, L]
    j = pos[None, :] - (lens - news)[:, None]                                           # place among the new tokens
    if s["tree"] is None:
        seen = j[:, None, :] <= i[None, :, None]
    else:
        seen = (s["tree"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1 == 1
        seen = seen & (j < 64)[:, None, :] | (j < 0)[:, None, :]
    seen = (seen & (pos[None, :] < lens[:, None])[:, None, :])[:, None, None]           # [S, 1, 1, n, L]
    sc = sc.unflatten(2, (g, n)).masked_fill(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (g, n))       # [S, H, G, n, D]
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)     # [S, n, Hq, D]
    return o[i[None, :] < news[:, None]].to(s["q"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import block_quantized_matmul_gb300 as qmm

        if op == "quantize":
            r, k, dt = case["rows"], case["k"], case["dtype"]
            qmm.qmm_mx4_quantize(dt, s["x"], r, k, k, s["codes"], s["scales"])
            qmm.qmm_mx4_dequantize(s["codes"], s["scales"], r, k, dt, s["y"], k)
            return s["y"]
        if op == "linear":
            m, k, n = case["m"], case["k"], case["n"]
            qmm.qmm_mx4_linear(s["w_codes"], s["w_scales"], k, n, case["dtype"], s["x"], k, m, case["out"], s["y"], n, s["ws"], s["ws"].numel())
            return s["y"]
        t, h, d, p, n = case["type"], case["heads"], case["d"], case["page"], s["count"]
        table, ld, seqs = s["pages"], s["pages"].shape[1], case["seqs"]
        if op == "cache":
            new, total, ld_tok = s["k"].shape[0], s["k_out"].shape[0], h * d
            qmm.qmm_cache_write(t, case["dtype"], s["k"], s["v"], ld_tok, ld_tok, new, h, d, s["slots"], s["k_cache"], s["v_cache"], n, p)
            qmm.qmm_cache_read(t, s["k_cache"], s["v_cache"], n, p, h, d, table, ld, s["starts"], seqs, total, case["dtype"], s["k_out"], s["v_out"], ld_tok, ld_tok)
            return {"k": s["k_out"], "v": s["v_out"]}
        hq, new = h * case["group"], s["q"].shape[0]
        qmm.qmm_cache_attend(t, s["k_cache"], s["v_cache"], n, p, h, d, table, ld, s["q_starts"], s["lens"], seqs, case["dtype"], s["q"], hq * d, new, hq,
                             s["tree"], s["scale"], case["new"], case["hi"], s["out"], hq * d, None, s["ws"], WORKSPACE)
        return s["out"]
    if op == "quantize":
        s["codes"], s["scales"] = _mx4_pack(*_mx4_codes(s["x"].float()))
        return _mx4_values(s["codes"], s["scales"]).to(s["x"].dtype)
    if op == "linear":
        x = _mx4_values(*_mx4_pack(*_mx4_codes(s["x"].float())))
        return (x @ _mx4_values(s["w_codes"], s["w_scales"]).t()).to(s["y"].dtype)
    return _plain_cache(s) if op == "cache" else _plain_attend(s)


# ---------------------------------------------------------------------------------- exact, in fp64
def _exact_mx4(x):
    """The MX4 values of rows, in fp64: every block on the grid of its own power of two."""
    r, k = x.shape
    b = x.double().view(-1, 32)
    top = b.abs().max(1, keepdim=True).values
    unit = torch.ldexp(torch.ones_like(top), (torch.frexp(top)[1] - 3).clamp(min=-127))
    u = b / unit
    # the spacing of E2M1 around u is 0.5 below 2, 1 below 4, 2 above
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0)).double()
    # torch.round takes ties to even multiples of the spacing, which are the even codes
    return ((torch.round(u / step) * step).clamp(-6, 6) * unit).view(r, k)


def _exact_operand(codes, scales, k):
    """An MX4 operand's values in fp64, found byte by byte through the layout's formula."""
    r = codes.shape[0]
    rr, bb = torch.arange(r, device="cuda")[:, None], torch.arange(k // 32, device="cuda")[None, :]
    at = (rr // 128 * -(-k // 128) + bb // 4) * 512 + rr % 32 * 16 + rr % 128 // 32 * 4 + bb % 4
    unit = torch.pow(2.0, scales[at].double() - 127)
    c = torch.empty(r, k, dtype=torch.uint8, device="cuda")
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    m = (c % 8).double()
    v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c < 8, v, -v) * unit.repeat_interleave(32, 1)


def _exact_block(t, x):
    """The q8_0 or q4_0 values of [..., D], in fp64 with the scale rounded to fp16."""
    b = x.double().reshape(-1, 32)
    if t == "q8_0":
        d = b.abs().max(1, keepdim=True).values / 127
        u = b / torch.where(d > 0, d, 1.0)
        q = torch.floor(u.abs() + 0.5) * torch.sign(u)
    else:
        hi, lo = b.max(1, keepdim=True), b.min(1, keepdim=True)
        tie = hi.values == -lo.values
        big = torch.where(hi.values > -lo.values, hi.values, lo.values)
        first = b.gather(1, torch.where(b.abs() == hi.values.abs(), torch.arange(32, device="cuda"), 31).min(1, keepdim=True).values)
        d = torch.where(tie, first, big) / -8
        u = b / torch.where(d != 0, d, 1.0)
        q = torch.where(d != 0, torch.floor(u + 8.5).clamp(0, 15) - 8, 0.0)
    return (q * d.to(torch.float16).double()).view(x.shape)


def _exact_tokens(cache, t, h, d, p, page, off):
    """fp64 [tokens][heads][D] from the bytes of a cache."""
    n, cb = d // 32, _code_bytes(t, d)
    base = (page[:, None] * h + torch.arange(h, device="cuda")[None, :]) * (p * _token_bytes(t, d))
    flat = cache.reshape(-1)
    e = torch.arange(d, device="cuda")
    at = base[:, :, None] + (off * cb)[:, None, None]
    if t == "q8_0":
        q = flat[at + e].double()
        q = torch.where(q > 127, q - 256, q)
    else:
        byte = flat[at + e // 32 * 16 + e % 16]
        q = torch.where(e % 32 < 16, byte % 16, byte // 16).double() - 8
    half = (base + p * cb)[:, :, None] + (off * 2 * n)[:, None, None] + 2 * torch.arange(n, device="cuda")
    s = torch.stack((flat[half], flat[half + 1]), -1).view(torch.float16).squeeze(-1).double()
    return q * s.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_mx4(s["x"])
    if op == "linear":
        return _exact_mx4(s["x"]) @ _exact_operand(s["w_codes"], s["w_scales"], case["k"]).t()
    t, h, d, p = case["type"], case["heads"], case["d"], case["page"]
    lens, news, table = _lens(case), _news(case), s["pages"].long()
    if op == "cache":
        out = {"k": [], "v": []}
        at = 0
        for i, (n, new) in enumerate(zip(lens, news)):
            pos = torch.arange(n - new, device="cuda")
            for name in out:
                old = _exact_tokens(s[name + "_cache"], t, h, d, p, table[i, pos // p], pos % p)
                out[name] += [old, _exact_block(t, s[name][at : at + new])]
            at += new
        return {name: torch.cat(v) for name, v in out.items()}
    outs, at, g = [], 0, case["group"]
    for i, (n, new) in enumerate(zip(lens, news)):
        if new == 0:
            continue
        pos = torch.arange(n, device="cuda")
        k, v = (_exact_tokens(s[name + "_cache"], t, h, d, p, table[i, pos // p], pos % p) for name in ("k", "v"))
        for r in range(new):
            seen = pos <= n - new + r
            if s["tree"] is not None:
                bits = int(s["tree"][at + r]) & (1 << 64) - 1
                allow = [True] * (n - new) + [bool(bits >> j & 1) for j in range(new)]
                seen = torch.tensor(allow, device="cuda")
            q = s["q"][at + r].double().view(h, g, d)
            w = torch.einsum("hgd,lhd->hgl", q, k[seen]) * s["scale"]
            outs.append(torch.einsum("hgl,lhd->hgd", torch.softmax(w, -1), v[seen]).reshape(h * g, d))
        at += new
    return torch.stack(outs) if outs else None
