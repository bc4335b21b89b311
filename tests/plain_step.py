"""Plain numpy forms (64-bit unless a rule fixes fp32 steps) of the plan, sparse-attention, norm and sampling calls, written from
their definitions in include/qmm.h, for the tests."""
from __future__ import annotations

import numpy as np

from tests import plain_ops as plain

f32 = np.float32


def up(a, b):
    return -(-a // b)


def plan(lens, news, P, pages, ring, ring_at, T):
    """Dict of all outputs; pages and ring as they are after the call."""
    pages, ring = pages.copy(), ring.copy()
    before = ring.copy()
    n_ring, ld = len(ring), pages.shape[1]
    first, last = (int(x) for x in ring_at)
    out = {"q_starts": [], "kv_lens": [], "next_lens": [], "slots": [-1] * T, "positions": [-1] * T}
    row, line, taken, back = 0, 0, 0, 0
    for s, (n, new) in enumerate(zip(lens, news)):
        n, new = min(max(int(n), 0), ld * P), int(new)
        out["q_starts"].append(row)
        held = up(n, P)
        if new < 0:
            for k in range(held):
                ring[(last + back) % n_ring] = pages[s, k]
                back += 1
            out["kv_lens"].append(0)
            out["next_lens"].append(0)
            continue
        need = up(n + new, P) - held if n + new <= ld * P else 0
        line += need
        run = n + new <= ld * P and row + new <= T and (need == 0 or line <= last - first)
        if run:
            for k in range(need):
                pages[s, held + k] = before[(first + taken) % n_ring]
                taken += 1
            for i in range(new):
                out["positions"][row + i] = n + i
                out["slots"][row + i] = int(pages[s, (n + i) // P]) * P + (n + i) % P
        out["kv_lens"].append(n + new if run else 0)
        out["next_lens"].append(n + new if run else n)
        row += new
    out["q_starts"].append(row)
    return {k: np.array(v) for k, v in out.items()} | {"pages": pages, "ring": ring, "next_at": np.array([first + taken, last + back])}


def up_half(x):
    """fp32 >= 0 rounded up to fp16."""
    h = x.astype(np.float16)
    return np.where(h.astype(f32) < x, np.nextafter(h, np.float16(np.inf)), h)


def bounds(type_, codes, scales):
    """Codes [P, bytes] and scales [P, D/32] of the keys of one page and head -> (lowest, highest: int8 [D], scales fp16 [D/32])."""
    v = plain.block_values(type_, codes, scales).reshape(len(codes), -1, 32)           # exact in fp64
    bad = ~np.isfinite(scales.astype(f32)).all(0)
    v = np.where(bad[None, :, None], 0.0, v)
    lo, hi = v.min(0).astype(f32), v.max(0).astype(f32)
    top = np.maximum(np.abs(lo), np.abs(hi)).max(-1)
    half = up_half(top / f32(127))
    d = np.where(half > 0, half.astype(f32), f32(1))[:, None]
    q = [np.clip(r(x / d), -127, 127).astype(np.int8).reshape(-1) for r, x in ((np.floor, lo), (np.ceil, hi))]
    return q[0], q[1], np.where(bad, np.float16(np.nan), half)


def bound_bytes(D):
    return up(2 * D + D // 32 * 2, 16) * 16


def q8_row(x):
    """fp32 [D] -> (codes fp64 [D], unrounded scales fp32 [D/32]; NaN scales where a block is not finite)."""
    b = x.astype(f32).reshape(-1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[:, None], f32(0), b)
    d = np.abs(b).max(-1) / f32(127)
    with np.errstate(all="ignore"):
        v = (b * np.where(d != 0, f32(1) / d, f32(0))[:, None]).astype(f32).astype(np.float64)
    v = np.where(np.isnan(v), 0, v)
    return np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127).reshape(-1), np.where(bad, f32(np.nan), d)


def score(q, lo, hi, d):
    """The fp32 score of one query row [D] and one page's bounds."""
    a, dq = q8_row(q)
    S = np.where(a > 0, a * hi, a * lo).reshape(-1, 32).sum(-1)
    s = f32(0)
    with np.errstate(all="ignore"):
        for b in range(len(S)):
            s = f32(s + f32(f32(dq[b] * f32(d[b])) * f32(S[b])))
    return s


def choose(scores, seen, always, budget):
    """scores [pages] (NaN counts as +inf), `seen` pages in question, set of those always chosen -> budget numbers, then -1."""
    key = np.where(np.isnan(scores), np.inf, scores)
    order = sorted(range(seen), key=lambda j: (j not in always, 0.0 if j in always else -key[j], j))
    pick = sorted(order[:budget])
    return pick + [-1] * (budget - len(pick))


def norm(x, h, w_post, gate, scale, w_pre, eps, round_h):
    """fp64 -> (h', y) for 2-d arrays; round_h rounds h' to its type."""
    if x is not None:
        x = x.astype(np.float64)
        if w_post is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w_post
        if gate is not None:
            x = x * gate
        h = h.astype(np.float64) + scale * x
    h = round_h(h)
    h64 = h.astype(np.float64)
    y = h64 / np.sqrt((h64 * h64).mean(-1, keepdims=True) + eps)
    return h, y if w_pre is None else y * w_pre


def sample(z, t, k, p, q, u):
    """(token, ln of its share, distance of u and top_p from the nearest border, as shares) of one row, in fp64."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    m = z.max()
    if m == -np.inf:
        return -1, -np.inf, 1.0
    order = np.argsort(-z, kind="stable")
    if not t > 0:
        return int(order[0]), 0.0, 1.0
    with np.errstate(all="ignore"):
        w = np.where(z == m, 1.0, np.exp((z - m) / t))
    w = np.where(np.isnan(w), 0.0, w)
    near = 1.0
    if 0 < k < len(z):
        order = order[:k]
    if p < 1:
        total = w[order].sum()
        before = np.cumsum(w[order]) - w[order]
        near = min(near, np.abs(before[1:] - p * total).min() / total if len(order) > 1 else 1.0)
        order = order[: max(1, int((before < p * total).sum()))]
    if q > 0:
        if q <= 1:
            near = min(near, np.abs(w[order][w[order] < 1] - q).min() if (w[order] < 1).any() else 1.0)
        order = order[: max(1, int((w[order] >= q).sum()))]
    kept = np.sort(order)
    upto = np.cumsum(w[kept])
    at = min(int((upto <= u * upto[-1]).sum()), len(kept) - 1)
    near = min(near, np.abs(upto / upto[-1] - u).min())
    return int(kept[at]), float(np.log(w[kept[at]] / upto[-1])), near
