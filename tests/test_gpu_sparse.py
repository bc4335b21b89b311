"""Sparse attention over the block-quantized cache on the GPU: the pages' bounds and the choice exactly, attention over the
chosen pages within the bound of the attention over all, against plain numpy forms."""
import math

import numpy as np
import pytest

from tests import plain_ops as plain
from tests import plain_step as step
from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, device, dtypes, random_tree, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


def starts_of(news):
    return np.concatenate(([0], np.cumsum(news))).astype(np.int32)


def gpu_bounds(c, news, lens=None, max_new=None, buf=None, T=None):
    import block_quantized_matmul_gb300 as qmm

    torch, lens = c.torch, c.lens if lens is None else lens
    if buf is None:
        buf = torch.full((c.n_pages, c.H, step.bound_bytes(c.D)), 0xA5, dtype=torch.uint8, device="cuda")
    qmm.qmm_cache_bounds(c.type, c.k_cache, c.n_pages, c.P, c.H, c.D, c.pages, c.table.shape[1], device(torch, starts_of(news)),
                         device(torch, np.array(lens, np.int32)), len(lens), int(sum(news)) if T is None else T, max(news) if max_new is None else max_new, buf)
    torch.cuda.synchronize()
    return buf


def plain_bounds(c, news, before, lens=None):
    """The whole buffer after the call."""
    out, D = before.copy(), c.D
    for s, (n, new) in enumerate(zip(c.lens if lens is None else lens, news)):
        if new == 0 or n == 0:
            continue
        for number in range(max(0, n - new) // c.P, (n - 1) // c.P + 1):
            page = c.table[s, number]
            if not 0 <= page < c.n_pages:
                continue
            have = min(c.P, n - number * c.P)
            for h in range(c.H):
                lo, hi, d = step.bounds(c.type, c.codes["k"][page, h, :have], c.scales["k"][page, h, :have])
                row = np.zeros(step.bound_bytes(D), np.uint8)
                row[:D], row[D : 2 * D] = lo.view(np.uint8), hi.view(np.uint8)
                row[2 * D : 2 * D + D // 16] = d.view(np.uint8)
                out[page, h] = row
    return out


def same_bounds(got, want, D):
    """Equal bytes; NaN scales alike."""
    g, w = got.copy(), want.copy()
    for a in (g, w):
        s = a[..., 2 * D : 2 * D + D // 16].copy().view(np.uint16)
        s[(s & 0x7FFF) > 0x7C00] = 0x7E00
        a[..., 2 * D : 2 * D + D // 16] = s.view(np.uint8)
    np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("lens,news,H,D,P", [
    ([1], [1], 1, 32, 16), ([16, 17, 0, 33], [1, 1, 0, 20], 2, 64, 16), ([300, 5, 64], [300, 5, 1], 3, 96, 128), ([100], [37], 8, 128, 64),
    ([70, 90], [70, 1], 1, 160, 32), ([50], [50], 2, 192, 16), ([40, 3], [2, 3], 1, 224, 32), ([600], [600], 2, 256, 256)])
def test_bounds(torch, type_, lens, news, H, D, P):
    c = Case(torch, type_, lens, H, D, P, seed=D).upload()
    buf = gpu_bounds(c, news)
    same_bounds(buf.cpu().numpy(), plain_bounds(c, news, np.full(buf.shape, 0xA5, np.uint8)), D)


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
def test_bounds_special_values(torch, type_):
    """Scales that are zero, subnormal, the largest, NaN and infinite, in their own blocks."""
    c = Case(torch, type_, [64], 1, 256, 64, seed=3)
    page = c.table[0, 0]
    s = c.scales["k"][page, 0]
    s[:, 0], s[:, 1], s[:, 2], s[5, 3], s[9, 4], s[:, 5] = 0, np.float16(6e-8), np.float16(65504), np.nan, -np.inf, np.float16(-65504)
    c.codes["k"][page, 0, 3] = 0x81                                  # -127 (Q8_0)
    c.upload()
    buf = gpu_bounds(c, [64])
    same_bounds(buf.cpu().numpy(), plain_bounds(c, [64], np.full(buf.shape, 0xA5, np.uint8)), 256)


def test_bounds_hold_the_keys(torch):
    """No key lies outside its page's bounds, but for half a step of fp32 in the divisions."""
    c = Case(torch, "q8_0", [500], 2, 128, 64, seed=4).upload()
    b = gpu_bounds(c, [500]).cpu().numpy()
    k = c.dense("k", 0)
    for i in range(500):
        row = b[c.table[0, i // 64]]
        d = row[:, 256:264].copy().view(np.float16).astype(np.float64).repeat(32, 1)
        lo, hi = (row[:, a : a + 128].view(np.int8) * d for a in (0, 128))
        assert (k[i] >= lo - 2.0 ** -23 * 128 * d).all() and (k[i] <= hi + 2.0 ** -23 * 128 * d).all()


def test_bounds_grow_with_the_sequence(torch):
    """Token by token (and max_new by max_new) the bounds become those of the whole; pages without new tokens stay."""
    n = 150
    c = Case(torch, "q8_0", [n], 2, 64, 16, seed=5).upload()
    whole = gpu_bounds(c, [n]).cpu().numpy()
    buf = None
    for i in range(1, n + 1):
        buf = gpu_bounds(c, [1], lens=[i], buf=buf)
    same_bounds(buf.cpu().numpy(), whole, 64)
    buf = None
    for i in (40, 41, 100, 150):
        buf = gpu_bounds(c, [40 if i != 100 else 59], lens=[i], buf=buf)
    same_bounds(buf.cpu().numpy(), whole, 64)
    last = gpu_bounds(c, [n], max_new=3).cpu().numpy()               # the pages of the last three tokens alone
    done = [c.table[0, k] for k in range((n - 3) // 16, (n - 1) // 16 + 1)]
    assert (last[[p for p in range(c.n_pages) if p not in done]] == 0xA5).all()
    same_bounds(last[done], whole[done], 64)


def test_bounds_leave_what_is_not_theirs(torch):
    """Pages out of the pool, sequences whose rows are not in q, and empty ones."""
    c = Case(torch, "q8_0", [40, 40, 40, 20], 1, 64, 16, seed=6)
    c.table[0, 1], c.table[1, 2] = -1, c.n_pages
    c.upload()
    buf = gpu_bounds(c, [40, 40, 0, 20], T=90)                       # the last sequence's rows pass T
    want = plain_bounds(c, [40, 40, 0, 0], np.full(buf.shape, 0xA5, np.uint8))
    same_bounds(buf.cpu().numpy(), want, 64)


# --------------------------------------------------------------------------------------------- choice
def gpu_select(c, bounds, q, news, dtype, tree, sinks, recent, budget, max_new=None, max_len=None, ldq=None, fill=-7, lens=None, stream=None, T=None):
    import block_quantized_matmul_gb300 as qmm

    torch = c.torch
    T_, Hq, D = q.shape
    T = T_ if T is None else T
    ldq = Hq * D if ldq is None else ldq
    qb = torch.full((T_, ldq), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    qb[:, : Hq * D] = device(torch, q.reshape(T_, -1)).to(dtypes(torch)[dtype])
    lens = c.lens if lens is None else lens
    max_new = max(news) if max_new is None else max_new
    max_len = max(lens) if max_len is None else max_len
    need = qmm.cache_select_workspace_size(T, c.H, c.P, max_len)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    chosen = torch.full((T_, c.H, budget), fill, dtype=torch.int32, device="cuda")
    qmm.qmm_cache_select(bounds, c.n_pages, c.P, c.H, D, c.pages, c.table.shape[1], device(torch, starts_of(news)), device(torch, np.array(lens, np.int32)),
                         len(lens), dtype, qb, ldq, T, Hq, tree, max_new, max_len, sinks, recent, budget, chosen, ws, need, stream=stream)
    torch.cuda.synchronize()
    return chosen, qb[:, : Hq * D].float().cpu().numpy().reshape(T_, Hq, D)


def plain_choice(c, bounds, q, news, tree, sinks, recent, budget, lens=None):
    b, D, G = bounds.cpu().numpy(), c.D, q.shape[1] // c.H
    out, at = [], 0
    for s, (n, new) in enumerate(zip(c.lens if lens is None else lens, news)):
        for i in range(new):
            first = n - new
            end = n - 1 if tree else first + i
            pages = end // c.P + 1 if end >= 0 else 0
            old = ((first if tree else first + i) // c.P if first + i >= 0 else 0) - recent + 1
            always = set(range(min(sinks, pages))) | set(range(max(0, old), pages))
            for h in range(c.H):
                scores = np.full(pages, -np.inf, np.float32)
                for number in range(pages if pages > budget else 0):
                    page = c.table[s, number]
                    if not 0 <= page < c.n_pages:
                        continue
                    row = b[page, h]
                    lo, hi, d = row[:D].view(np.int8).astype(int), row[D : 2 * D].view(np.int8).astype(int), row[2 * D : 2 * D + D // 16].copy().view(np.float16)
                    best = [step.score(q[at + i, h * G + g], lo, hi, d.astype(np.float32)) for g in range(G)]
                    scores[number] = np.inf if np.isnan(best).any() else max(best)
                out.append(step.choose(scores, pages, always, budget))
        at += new
    return np.array(out, np.int32).reshape(at, c.H, budget)


SELECT = [
    # lens, news, H, G, D, P, sinks, recent, budget
    ([1], [1], 1, 1, 64, 16, 0, 1, 1), ([500], [1], 2, 4, 128, 16, 1, 2, 6), ([0, 16, 17, 33, 400, 64], [0, 1, 1, 1, 1, 1], 2, 3, 64, 16, 1, 1, 4),
    ([700, 90], [1, 1], 1, 8, 96, 32, 0, 1, 3), ([300], [1], 1, 16, 256, 16, 2, 3, 8), ([410, 333], [5, 2], 2, 2, 160, 16, 1, 2, 7),
    ([250], [40], 1, 4, 32, 16, 1, 1, 5), ([300, 280], [9, 20], 1, 7, 192, 16, 0, 2, 9), ([200], [1], 1, 64, 32, 16, 1, 1, 4), ([260, 20], [3, 3], 2, 1, 224, 16, 3, 1, 8),
]


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("lens,news,H,G,D,P,sinks,recent,budget", SELECT)
def test_select(torch, type_, dtype, tree, lens, news, H, G, D, P, sinks, recent, budget):
    c = Case(torch, type_, lens, H, D, P, seed=D).upload()
    bounds = gpu_bounds(c, lens)
    budget += (max(news) + P - 2) // P if tree else 0
    rng = np.random.default_rng(D)
    q = rng.standard_normal((sum(news), H * G, D)).astype(np.float32)
    words = device(torch, random_tree(rng, news).view(np.int64)) if tree else None
    chosen, q = gpu_select(c, bounds, q, news, dtype, words, sinks, recent, budget)
    np.testing.assert_array_equal(chosen.cpu().numpy(), plain_choice(c, bounds, q, news, tree, sinks, recent, budget))


def test_select_ties_infinities_and_pages_out_of_the_pool(torch):
    """Pages alike give scores alike: the earlier ones are chosen.  A page with a NaN scale comes before all others, one out of
    the pool behind them."""
    P, D, n = 16, 64, 16 * 40
    c = Case(torch, "q8_0", [n], 1, D, P, seed=8)
    for number in range(0, 40, 3):
        c.codes["k"][c.table[0, number]] = c.codes["k"][c.table[0, 0]]
        c.scales["k"][c.table[0, number]] = c.scales["k"][c.table[0, 0]]
    c.scales["k"][c.table[0, 20], 0, 3, 1] = np.nan
    c.table[0, 22] = c.n_pages + 3
    c.upload()
    bounds = gpu_bounds(c, [n])
    q = np.random.default_rng(9).standard_normal((1, 4, D)).astype(np.float32)
    for budget in (2, 3, 5, 9, 14, 20, 38, 39):
        chosen, qr = gpu_select(c, bounds, q, [1], "bf16", None, 0, 1, budget)
        want = plain_choice(c, bounds, qr, [1], False, 0, 1, budget)
        np.testing.assert_array_equal(chosen.cpu().numpy(), want)
        assert 20 in want and (22 in want) == (budget >= 40)
    zero, qr = gpu_select(c, bounds, 0 * q, [1], "f16", None, 0, 1, 4)              # every score is 0, but the NaN one
    assert zero.tolist() == [[[0, 1, 20, 39]]]
    q[0, 1, 5] = np.inf                                                             # every score is NaN: the earliest pages
    bad, qr = gpu_select(c, bounds, q, [1], "f16", None, 0, 1, 4)
    assert bad.tolist() == [[[0, 1, 2, 39]]]


def test_select_leaves_rows_that_are_not_its_own(torch):
    """Rows before the first and behind the last sequence, past max_new, and of sequences not all in q keep what they hold; a sequence longer
    than max_len, or without tokens, gets no page."""
    lens, news = [200, 64, 300], [4, 4, 4]
    c = Case(torch, "q8_0", lens, 1, 64, 16, seed=10).upload()
    bounds = gpu_bounds(c, lens)
    q = np.random.default_rng(11).standard_normal((14, 2, 64)).astype(np.float32)
    chosen, qr = gpu_select(c, bounds, q, news, "bf16", None, 1, 1, 4, max_new=3)
    want = plain_choice(c, bounds, qr, news, False, 1, 1, 4)
    got = chosen.cpu().numpy()
    for i in range(14):
        np.testing.assert_array_equal(got[i], np.full((1, 4), -7) if i >= 12 or i % 4 == 3 else want[i])
    got = gpu_select(c, bounds, q, news, "bf16", None, 1, 1, 4, max_len=200)[0].cpu().numpy()
    np.testing.assert_array_equal(got[:8], want[:8])
    assert (got[8:12] == -1).all() and (got[12:] == -7).all()
    got = gpu_select(c, bounds, q, news, "bf16", None, 1, 1, 4, lens=[200, 0, 300])[0].cpu().numpy()
    assert (got[4:8] == -1).all()
    got = gpu_select(c, bounds, q, news, "bf16", None, 1, 1, 4, T=11)[0].cpu().numpy()
    np.testing.assert_array_equal(got[:8], want[:8])
    assert (got[8:] == -7).all()


def test_select_strided_queries_and_streams(torch):
    lens, news = [1000, 777], [1, 1]
    c = Case(torch, "q4_0", lens, 2, 128, 32, seed=12).upload()
    bounds = gpu_bounds(c, lens)
    q = np.random.default_rng(13).standard_normal((2, 8, 128)).astype(np.float32)
    a, _ = gpu_select(c, bounds, q, news, "f16", None, 1, 2, 8)
    b, _ = gpu_select(c, bounds, q, news, "f16", None, 1, 2, 8, ldq=1024 + 24, stream=torch.cuda.Stream(), max_len=5000)
    assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ attention
def gpu_attend(c, q, news, dtype, tree, scale, chosen, workspace=None, ldq=None, lse=True, lens=None, stream=None, T=None):
    import block_quantized_matmul_gb300 as qmm

    torch = c.torch
    T_, Hq, D = q.shape
    T = T_ if T is None else T
    ldq = Hq * D if ldq is None else ldq
    qb = torch.full((T_, ldq), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    qb[:, : Hq * D] = device(torch, q.reshape(T_, -1)).to(dtypes(torch)[dtype])
    ob = torch.full((T_, ldq), -7.0, dtype=dtypes(torch)[dtype], device="cuda")
    lb = torch.full((T_, Hq), -7.0, device="cuda") if lse else None
    budget = chosen.shape[2]
    lens = c.lens if lens is None else lens
    if workspace is None:
        workspace = qmm.cache_attend_chosen_workspace_size(T, c.H, Hq, D, c.P, budget)
    ws = torch.full((max(1, workspace),), 0xFF, dtype=torch.uint8, device="cuda") if workspace else None
    td = device(torch, tree.astype(np.uint64).view(np.int64)) if tree is not None else None
    qmm.qmm_cache_attend_chosen(c.type, c.k_cache, c.v_cache, c.n_pages, c.P, c.H, D, c.pages, c.table.shape[1], device(torch, starts_of(news)),
                                device(torch, np.array(lens, np.int32)), len(lens), dtype, qb, ldq, T, Hq, td, scale, chosen, budget, ob, ldq, lb, ws,
                                workspace, stream=stream)
    torch.cuda.synchronize()
    assert (ob[:, Hq * D:] == -7).all()
    return ob[:, : Hq * D].float().cpu().numpy().reshape(T_, Hq, D), None if lb is None else lb.cpu().numpy(), \
        qb[:, : Hq * D].float().cpu().numpy().reshape(T_, Hq, D)


def check_attend(c, got, lse, q, news, tree, scale, dtype, chosen, lens=None):
    """As for the attention over all (test_gpu_cache.check_attend), over the keys of the chosen pages, each as often as listed."""
    G, at = q.shape[1] // c.H, 0
    for s, (n, new) in enumerate(zip(c.lens if lens is None else lens, news)):
        seen_all = visible(n, new, tree, at)
        k, v = c.dense("k", s)[:n], c.dense("v", s)[:n]
        for i in range(new):
            for h in range(c.H):
                keys = []
                for number in chosen[at + i, h]:
                    if number < 0:
                        break
                    if number < c.table.shape[1] and 0 <= c.table[s, number] < c.n_pages:
                        keys += [j for j in range(int(number) * c.P, min(n, int(number) * c.P + c.P)) if seen_all[i, j]]
                keys = np.array(keys, int)
                for g in range(G):
                    hq = h * G + g
                    out, mag, ls, big = plain.attend(q[at + i : at + i + 1, hq].astype(np.float64), k[keys][:, h], v[keys][:, h], np.ones((1, len(keys)), bool), scale)
                    tol = (2.0 ** -9 + 2.0 ** -20 * big[:, None]) * mag + plain.ULP[dtype] * np.abs(out) + 1e-6
                    r = got[at + i, hq][None]
                    np.testing.assert_array_equal(np.isnan(r), np.isnan(out))
                    err = np.abs(np.nan_to_num(r) - np.nan_to_num(out))
                    assert (err <= np.nan_to_num(tol, nan=1e9)).all(), (s, i, hq, float(err.max()))
                    if lse is not None:
                        if len(keys) == 0:
                            assert np.isneginf(lse[at + i, hq]) and (r == 0).all()
                        elif np.isfinite(ls[0]):
                            assert abs(lse[at + i, hq] - ls[0]) <= 1e-5 + 2.0 ** -20 * big[0]
        at += new


ATTEND = SELECT + [([130, 64], [3, 30], 1, 16, 128, 16, 1, 1, 4), ([257], [2], 1, 33, 64, 32, 0, 1, 4), ([90], [1], 1, 64, 128, 16, 0, 1, 3), ([100], [1], 1, 40, 256, 16, 0, 1, 3)]


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("lens,news,H,G,D,P,sinks,recent,budget", ATTEND)
def test_attend_over_the_choice(torch, type_, dtype, tree, lens, news, H, G, D, P, sinks, recent, budget):
    c = Case(torch, type_, lens, H, D, P, seed=D).upload()
    bounds = gpu_bounds(c, lens)
    budget += (max(news) + P - 2) // P if tree else 0
    rng = np.random.default_rng(D + 1)
    q = rng.standard_normal((sum(news), H * G, D)).astype(np.float32)
    words = random_tree(rng, news) if tree else None
    chosen, q = gpu_select(c, bounds, q, news, dtype, device(torch, words.view(np.int64)) if tree else None, sinks, recent, budget)
    got, lse, q = gpu_attend(c, q, news, dtype, words, 1 / math.sqrt(D), chosen)
    check_attend(c, got, lse, q, news, words, 1 / math.sqrt(D), dtype, chosen.cpu().numpy())


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("workspace", [0, 4096, 200000, None, 64 << 20])
def test_attend_any_list_and_any_workspace(torch, type_, workspace):
    """Lists out of order, with pages twice, past the end, out of the table, ended early, empty, full."""
    lens, news, budget = [900, 37, 0], [2, 2, 1], 40
    c = Case(torch, type_, lens, 2, 64, 16, seed=20)
    c.table[0, 7] = -1
    c.upload()
    rng = np.random.default_rng(21)
    chosen = rng.integers(0, 57, (5, 2, budget)).astype(np.int32)
    chosen[0, 0, 5:] = -1
    chosen[0, 1] = -1
    chosen[1, 0, 3], chosen[1, 0, 9] = 1 << 30, 2147483647
    chosen[1, 1, 1] = -2147483648
    chosen[2, 0, 0] = 0
    q = rng.standard_normal((5, 8, 64)).astype(np.float32)
    got, lse, q = gpu_attend(c, q, news, "f16", None, 0.2, device(torch, chosen), workspace=workspace)
    check_attend(c, got, lse, q, news, None, 0.2, "f16", chosen)
    again, _, _ = gpu_attend(c, q, news, "f16", None, 0.2, device(torch, chosen), workspace=workspace, lse=False, ldq=600, stream=torch.cuda.Stream())
    np.testing.assert_array_equal(got, again)


def test_all_pages_chosen_is_the_attention_over_all(torch):
    from tests.test_gpu_cache import run_attend

    lens, news = [1500, 200], [1, 3]
    c = Case(torch, "q8_0", lens, 2, 128, 64, seed=22).upload()
    q = np.random.default_rng(23).standard_normal((4, 8, 128)).astype(np.float32)
    chosen = np.full((4, 2, 30), -1, np.int32)
    chosen[0, :, :24], chosen[1:, :, :4] = np.arange(24), np.arange(4)
    got, lse, qr = gpu_attend(c, q, news, "f16", None, 0.1, device(torch, chosen))
    want, wl, _ = run_attend(c, q, starts_of(news), lens, "f16", None, 0.1)
    # two sums of the same terms in another order, each rounded to fp16 at the end
    assert (np.abs(got - want) <= 2.0 ** -9 * np.abs(want).max()).all() and (np.abs(lse - wl) <= 1e-5).all()


def test_attend_nan_and_infinity_reach_only_who_sees_them(torch):
    """Values that are not finite in tokens behind the row's own, outside its tree, and in pages that it did not choose."""
    lens, news, P = [200, 100], [3, 4], 16
    c = Case(torch, "q8_0", lens, 1, 128, P, seed=24)
    for s, pos, name, block, v in ((0, 199, "v", 1, np.nan), (0, 198, "k", 0, np.nan), (0, 50, "v", 2, np.inf), (1, 97, "v", 3, np.nan), (1, 98, "k", 1, np.inf)):
        c.scales[name][c.table[s, pos // P], 0, pos % P, block] = v
        c.codes[name][c.table[s, pos // P], 0, pos % P, 32 * block : 32 * block + 32] |= 1      # (no 0 * inf)
    c.upload()
    tree = np.array([1 << i for i in range(3)] + [1 << i for i in range(4)], np.uint64)
    chosen = np.full((7, 1, 6), -1, np.int32)
    chosen[:, 0, :3] = [0, 1, 12]
    chosen[1, 0, 3] = 3                                                                             # place 50 is there
    chosen[3:, 0, :3] = [0, 5, 6]
    q = np.random.default_rng(25).standard_normal((7, 2, 128)).astype(np.float32)
    for words in (None, tree):
        got, lse, qr = gpu_attend(c, q, news, "bf16", words, 0.1, device(torch, chosen))
        with np.errstate(invalid="ignore"):
            check_attend(c, got, None, qr, news, words, 0.1, "bf16", chosen)
        assert np.isfinite(got[0]).all() and np.isfinite(got[3]).all() and not np.isfinite(got[1]).all()


def test_attend_skips_what_is_not_its_own(torch):
    """Rows behind the last sequence and of sequences not all in q stay; rows of a sequence that waits (length 0) are 0."""
    lens, news = [100, 90, 80], [2, 2, 2]
    c = Case(torch, "q8_0", lens, 1, 64, 16, seed=26).upload()
    q = np.random.default_rng(27).standard_normal((8, 4, 64)).astype(np.float32)
    chosen = device(torch, np.tile(np.arange(5, dtype=np.int32), (8, 1, 1)))
    got, lse, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen)
    assert (got[6:] == -7).all() and (lse[6:] == -7).all() and (got[:6] != -7).all()
    got, lse, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen, T=5)
    assert (got[4:] == -7).all() and (lse[4:] == -7).all() and (got[:4] != -7).all()
    got, lse, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen, lens=[100, 0, 80])
    assert (got[2:4] == 0).all() and np.isneginf(lse[2:4]).all() and (got[4:6] != 0).any()


@pytest.mark.parametrize("workspace", [None, 0])
def test_attend_long_lists(torch, workspace):
    """One token over lists of thousands of keys, split over the GPU and not."""
    n, P, budget = 60000, 64, 300
    c = Case(torch, "q8_0", [n], 2, 128, P, seed=28).upload()
    bounds = gpu_bounds(c, [n])
    q = 2 * np.random.default_rng(29).standard_normal((1, 8, 128)).astype(np.float32)
    chosen, _ = gpu_select(c, bounds, q, [1], "f16", None, 1, 4, budget)
    assert (chosen >= 0).all() and (chosen[..., 1:] > chosen[..., :-1]).all()
    got, lse, qr = gpu_attend(c, q, [1], "f16", None, 0.1, chosen, workspace=workspace)
    check_attend(c, got, lse, qr, [1], None, 0.1, "f16", chosen.cpu().numpy())
