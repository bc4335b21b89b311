"""The choice of pages at real lengths, against a plain form over all pages at once: several CTAs and turns along the pages, tiles that
hold tokens of several sequences, more pages than stay in registers, and scores so alike that the border is narrowed down over several
rounds.  Bounds are random bytes, no cache is needed."""
import numpy as np
import pytest

from tests import plain_step as step
from tests.test_gpu_cache import Case, device
from tests.test_gpu_sparse import gpu_bounds, gpu_select, torch  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
f32 = np.float32


class Pages:
    """A table of distinct pages (a few entries out of the pool) and their bounds."""

    def __init__(self, torch, rng, lens, H, D, P, kind, out_of_pool=0.01):
        self.torch, self.lens, self.H, self.D, self.P = torch, lens, H, D, P
        most = max(1, max(-(-n // P) for n in lens))
        self.n_pages = len(lens) * most + 3
        self.table = rng.permutation(self.n_pages)[: len(lens) * most].reshape(len(lens), most).astype(np.int32)
        n, db = self.n_pages, D // 32
        a, b = (rng.integers(-127, 128, (n, H, D), dtype=np.int8) for _ in range(2))
        self.lo, self.hi = np.minimum(a, b), np.maximum(a, b)
        self.d = rng.uniform(0.5, 2, (n, H, db)).astype(np.float16)
        if kind in ("alike", "near", "far"):
            # all pages' bounds are one page's; near: but for three elements of a block whose scale is small; far: and a few pages stand out
            self.lo[:], self.hi[:], self.d[:] = self.lo[0], self.hi[0], self.d[0]
            if kind != "alike":
                self.d[..., -1] = 2.0 ** -10
                for e in (D - 5, D - 9, D - 20):
                    self.lo[..., e] = rng.integers(-127, 1, (n, H))
                    self.hi[..., e] = rng.integers(0, 128, (n, H))
            if kind == "far":
                some = rng.random((n, H)) < 0.002
                self.d[some] *= 100
        elif kind == "levels":
            self.d[:] = rng.choice([0.25, 1, 1.001953125, 60], (n, H, 1), p=[0.3, 0.4, 0.29, 0.01])
            self.lo[:], self.hi[:] = self.lo[0], self.hi[0]
        elif kind == "nan":
            self.d[rng.random((n, H)) < 0.1, 0] = np.nan
            self.d[rng.random((n, H)) < 0.1] = 0
        raw = np.zeros((n, H, step.bound_bytes(D)), np.uint8)
        raw[..., :D], raw[..., D : 2 * D] = self.lo.view(np.uint8), self.hi.view(np.uint8)
        raw[..., 2 * D : 2 * D + 2 * db] = self.d.view(np.uint8)
        self.bounds = device(torch, raw)
        gone = rng.random(self.table.shape) < out_of_pool
        self.table[gone] = rng.choice([-1, self.n_pages, 1 << 30], int(gone.sum()))
        self.pages = device(torch, self.table)


def read_bounds(c, raw):
    """Of a Case, whose bounds the library wrote."""
    D = c.D
    c.lo, c.hi = raw[..., :D].copy().view(np.int8), raw[..., D : 2 * D].copy().view(np.int8)
    c.d = raw[..., 2 * D : 2 * D + D // 16].copy().view(np.float16)


def plain_choice(c, q, news, tree, sinks, recent, budget):
    D, G, H, db = c.D, q.shape[1] // c.H, c.H, c.D // 32
    codes, scales = (np.array(x) for x in zip(*(step.q8_row(r) for r in q.reshape(-1, D))))
    codes, scales = codes.reshape(len(q), H, G, db, 32), scales.reshape(len(q), H, G, db).astype(f32)
    out, at = np.full((len(q), H, budget), -1, np.int32), 0
    for s, (n, new) in enumerate(zip(c.lens, news)):
        pages = -(-n // c.P)
        ids = c.table[s, :pages]
        there = (ids >= 0) & (ids < c.n_pages)
        ids = np.where(there, ids, 0)
        for h in range(H if new else 0):
            lo, hi = (x[ids, h].reshape(pages, db, 32).astype(np.float64) for x in (c.lo, c.hi))
            a = codes[at : at + new, h]                                               # [new, G, db, 32]
            S = np.einsum("tgbe,pbe->tgpb", np.maximum(a, 0), hi, optimize=True) + np.einsum("tgbe,pbe->tgpb", np.minimum(a, 0), lo, optimize=True)
            score = np.zeros((new, G, pages), f32)
            with np.errstate(all="ignore"):
                for b in range(db):
                    score = score + (scales[at : at + new, h, :, None, b] * c.d[ids, h, b].astype(f32)) * S[..., b].astype(f32)
            score = np.where(np.isnan(score), f32(np.inf), score).max(1)
            score = np.where(there, score, f32(-np.inf))
            for i in range(new):
                first = n - new
                last = n - 1 if tree else first + i
                seen = last // c.P + 1
                old = (first if tree else last) // c.P - recent + 1
                j = np.arange(seen)
                always = (j < sinks) | (j >= old)
                pick = np.sort(np.lexsort((j, np.where(always, 0, -score[i, :seen]), ~always))[:budget])
                out[at + i, h, : len(pick)] = pick
        at += new
    return out


def check(torch, rng, lens, news, H, G, D, P, kind, sinks, recent, budgets, dtype="bf16", tree=False, max_len=None):
    c = Pages(torch, rng, lens, H, D, P, kind)
    q = rng.standard_normal((sum(news), H * G, D)).astype(f32)
    words = torch.ones(sum(news), dtype=torch.int64, device="cuda") if tree else None
    for budget in budgets:
        budget += (max(news) + P - 2) // P if tree else 0
        got, qr = gpu_select(c, c.bounds, q, news, dtype, words, sinks, recent, budget, max_len=max_len)
        np.testing.assert_array_equal(got.cpu().numpy(), plain_choice(c, qr, news, tree, sinks, recent, budget))


KINDS = ["random", "alike", "near", "far", "levels", "nan"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,D", [(4, 128), (1, 64), (16, 96)])
def test_one_token_over_thousands_of_pages(torch, kind, G, D):  # noqa: F811
    check(torch, np.random.default_rng(1), [64000, 40001], [1, 1], 2, G, D, 16, kind, 1, 4, [6, 32, 300, 2500, 3999])


@pytest.mark.parametrize("kind", KINDS)
def test_more_pages_than_stay_in_registers(torch, kind):  # noqa: F811
    """4097 pages and more, and shorter sequences beside them."""
    check(torch, np.random.default_rng(2), [65537, 81234, 65536, 300, 4096 * 16 + 16], [1] * 5, 1, 2, 64, 16, kind, 2, 3, [8, 64, 1000, 4096])
    check(torch, np.random.default_rng(3), [150000], [3], 2, 1, 32, 16, kind, 0, 1, [1, 40, 5000])


@pytest.mark.parametrize("kind", ["random", "near", "nan"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
def test_several_turns_of_pages(torch, kind, tree):  # noqa: F811
    """So many rows that a CTA goes on from 64 pages to others: one sequence's tokens, and tiles with tokens of several."""
    rng = np.random.default_rng(4)
    check(torch, rng, [30000], [40], 8, 2, 64, 16, kind, 1, 2, [5, 100], tree=tree)
    check(torch, rng, [20000, 30000, 900, 26000, 0, 64], [5, 30, 11, 2, 0, 3], 8, 1, 64, 16, kind, 1, 2, [5, 100], tree=tree)
    check(torch, rng, [30000 - 500 * i for i in range(57)], [2] + [1] * 56, 4, 3, 32, 16, kind, 0, 1, [7], tree=tree)


@pytest.mark.parametrize("D", [32, 160, 192, 224, 256])
def test_several_turns_of_pages_of_every_width(torch, D):  # noqa: F811
    rng = np.random.default_rng(5)
    check(torch, rng, [12000, 14000, 3000], [17, 9, 30], 6, 4, D, 16, "random", 1, 2, [9], dtype="f16")
    check(torch, rng, [5000 + 40 * i for i in range(30)], [1] * 30, 8, 8, D, 16, "random", 1, 2, [9])


def test_single_tokens_of_many_sequences(torch):  # noqa: F811
    """One token a CTA, and all its pages in turns."""
    rng = np.random.default_rng(6)
    check(torch, rng, [int(n) for n in rng.integers(0, 6000, 600)], [1] * 600, 1, 2, 32, 16, "random", 1, 1, [12], max_len=20000)


def test_a_long_sequence_of_keys(torch):  # noqa: F811
    """The bounds that the library wrote of 60000 keys."""
    n, P = 60000, 64
    c = Case(torch, "q8_0", [n], 2, 128, P, seed=28).upload()
    bounds = gpu_bounds(c, [n])
    read_bounds(c, bounds.cpu().numpy())
    q = 2 * np.random.default_rng(29).standard_normal((1, 8, 128)).astype(f32)
    for budget in (20, 300, 900):
        chosen, qr = gpu_select(c, bounds, q, [1], "f16", None, 1, 4, budget)
        np.testing.assert_array_equal(chosen.cpu().numpy(), plain_choice(c, qr, [1], False, 1, 4, budget))
