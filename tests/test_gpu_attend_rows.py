"""Attention over the block-quantized cache with many rows a sequence (32 on mma, 128 on tcgen05): the cases in
which a row sees nothing, sees infinities or NaN that others do not, or pages end inside a tile."""
import math

import numpy as np
import pytest

from tests import plain_ops as plain
from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, check_attend, device, random_tree, run_attend

pytestmark = pytest.mark.gpu

ROWS = [(10, 2, 64), (24, 2, 128), (40, 4, 96), (64, 3, 32), (16, 2, 256)]      # new tokens, query heads a head, elements


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


@pytest.mark.parametrize("type_,dtype", [("q8_0", "bf16"), ("q4_0", "f16")])
@pytest.mark.parametrize("new,G,D", ROWS)
def test_rows_that_see_nothing(torch, type_, dtype, new, G, D):
    lens, news = [new, 100 + new, 0], [new, new, 0]
    c = Case(torch, type_, lens, 2, D, 16).upload()
    q_starts = np.array([0, new, 2 * new, 2 * new])
    tree = random_tree(np.random.default_rng(3), news)
    tree[new - 1] = tree[3] = 0            # sequence 0 has no context: the rows see nothing
    tree[new + 2] = 0                      # sequence 1 has: the row sees the context alone
    q = np.random.default_rng(4).standard_normal((2 * new, 2 * G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, dtype, tree, 1 / math.sqrt(D))
    for i in (3, new - 1):
        assert (got[i] == 0).all() and np.isneginf(lse[i]).all()
    check_attend(c, got, lse, q, q_starts, lens, tree, 1 / math.sqrt(D), dtype)


@pytest.mark.parametrize("type_,dtype", [("q8_0", "bf16"), ("q4_0", "f16")])
@pytest.mark.parametrize("new,G,D", ROWS)
def test_nan_and_infinity_reach_only_who_sees_them(torch, type_, dtype, new, G, D):
    lens, news = [50 + new, 300 + new], [new, new]
    c = Case(torch, type_, lens, 1, D, 16)
    q_starts = np.array([0, new, 2 * new])
    tree = np.array([1 << i for i in range(new)] * 2, dtype=np.uint64)          # each new token sees itself and the context
    blocks = D // 32
    for s, n in enumerate(lens):
        for b, name, block, value in ((2, "v", blocks - 1, np.nan), (5, "k", blocks // 2, np.nan), (6, "v", 0, np.inf)):
            pos = n - new + b
            c.scales[name][c.table[s, pos // 16], 0, pos % 16, block] = value
            if value == np.inf:
                # codes that are not 0, so that no product is 0 * inf
                at = slice(0, 32) if type_ == "q8_0" else slice(0, 16)
                c.codes[name][c.table[s, pos // 16], 0, pos % 16, at] = 0x11
    c.upload()
    q = np.random.default_rng(5).standard_normal((2 * new, G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, dtype, tree, 0.1)
    for base in (0, new):
        bad = ~np.isfinite(got[base:base + new])
        assert bad[2, :, D - 32:].all() and bad[5].all() and bad[6, :, :32].all()
        assert bad.sum() == G * (32 + D + 32)
    for name in "kv":                      # the same without them, for the other rows
        c.scales[name] = np.where(np.isfinite(c.scales[name]), c.scales[name], np.float16(0.01))
    clean, _, _ = run_attend(c.upload(), q, q_starts, lens, dtype, tree, 0.1)
    for base in (0, new):
        for i in (0, 1, 3, 4, 7):
            np.testing.assert_array_equal(got[base + i], clean[base + i])


@pytest.mark.parametrize("new,G,D", ROWS)
def test_pages_out_of_the_pool_are_not_seen(torch, new, G, D):
    lens = [200 + new, 80 + new]
    c = Case(torch, "q8_0", lens, 1, D, 16).upload()
    q = np.random.default_rng(7).standard_normal((2 * new, G, D)).astype(np.float32)
    table = c.table.copy()
    c.table[0, 1], c.table[0, 9], c.table[1, 0] = -1, c.n_pages + 5, -7
    c.pages = device(torch, c.table)
    got, lse, q = run_attend(c, q, np.array([0, new, 2 * new]), lens, "bf16", None, 0.125)
    c.table = table
    for s, hidden in ((0, (1, 9)), (1, (0,))):
        n = lens[s]
        seen = np.arange(n)[None, :] <= (n - new + np.arange(new))[:, None]
        for page in hidden:
            seen[:, 16 * page:16 * page + 16] = False
        for hq in range(G):
            out, mag, ls, big = plain.attend(q[s * new:(s + 1) * new, hq].astype(np.float64), c.dense("k", s)[:, 0], c.dense("v", s)[:, 0], seen, 0.125)
            tol = (2.0 ** -9 + 2.0 ** -20 * big[:, None]) * mag + 2.0 ** -8 * np.abs(out) + 1e-6
            assert (np.abs(got[s * new:(s + 1) * new, hq] - out) <= tol).all()
            assert (np.abs(lse[s * new:(s + 1) * new, hq] - ls) <= 1e-5 + 2.0 ** -20 * big).all()


@pytest.mark.parametrize("workspace", [0, None])
@pytest.mark.parametrize("new,G,D", [(24, 2, 128), (10, 2, 128), (130, 4, 64)])
def test_long_sequences_split_or_not(torch, new, G, D, workspace):
    lens, news = [3001 + new, 257], [new, min(new, 100)]
    c = Case(torch, "q8_0", lens, 1, D, 64).upload()
    q_starts = np.concatenate(([0], np.cumsum(news)))
    q = 3 * np.random.default_rng(2).standard_normal((q_starts[-1], G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.3, workspace=workspace)
    check_attend(c, got, lse, q, q_starts, lens, None, 0.3, "bf16")
    again, _, _ = run_attend(c, q, q_starts, lens, "bf16", None, 0.3, workspace=workspace, lse=False)
    np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_scores_and_small_values(torch, dtype):
    """Scores that grow by hundreds from tile to tile (the outputs so far are scaled down each time), values around
    1e-4, queries of mixed size."""
    lens, new, G, D = [900], 20, 4, 64
    c = Case(torch, "q8_0", lens, 1, D, 64, key_scale=0.5)
    for i, page in enumerate(c.table[0]):
        c.scales["k"][page] = (c.scales["k"][page].astype(np.float32) * (1 + i)).astype(np.float16)
    c.scales["v"] = (c.scales["v"].astype(np.float32) * 1e-4).astype(np.float16)
    c.upload()
    q = np.random.default_rng(6).standard_normal((new, G, D)).astype(np.float32) * np.array([1e-3, 1, 10, 100], np.float32)[None, :, None]
    got, lse, q = run_attend(c, q, np.array([0, new]), lens, dtype, None, 0.125)
    k, v = c.dense("k", 0)[:, 0], c.dense("v", 0)[:, 0]
    seen = np.arange(900)[None, :] <= (900 - new + np.arange(new))[:, None]
    for hq in range(G):
        out, mag, ls, big = plain.attend(q[:, hq].astype(np.float64), k, v, seen, 0.125)
        # the last term: half the smallest step of an fp16 output
        tol = (2.0 ** -9 + 2.0 ** -20 * big[:, None]) * mag + plain.ULP[dtype] * np.abs(out) + 1e-9 + (2.0 ** -25 if dtype == "f16" else 0.0)
        assert (np.abs(got[:, hq] - out) <= tol).all(), hq


def test_first_tokens_of_a_sequence(torch):
    """A prompt whose tokens are all new, of a length inside a tile, and one that ends with a page."""
    for lens in ([1, 127], [128, 129], [64, 300]):
        c = Case(torch, "q4_0", lens, 2, 128, 32).upload()
        q_starts = np.concatenate(([0], np.cumsum(lens)))
        q = np.random.default_rng(8).standard_normal((q_starts[-1], 4, 128)).astype(np.float32)
        got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.088)
        check_attend(c, got, lse, q, q_starts, lens, None, 0.088, "bf16")
