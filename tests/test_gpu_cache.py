"""The block-quantized key/value cache on the GPU: written bytes and read values exactly, attention within its
bound, against plain numpy forms in 64 bits."""
import math

import numpy as np
import pytest

from tests import plain_ops as plain
from tests.gpu_util import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


def dtypes(torch):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def device(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,P,pad", [(1, 1, 32, 16, 0), (5, 2, 64, 16, 0), (33, 8, 128, 64, 0), (70, 3, 96, 32, 8), (9, 2, 256, 256, 3)])
def test_write_bytes(torch, type_, dtype, T, H, D, P, pad):
    import block_quantized_matmul_gb300 as qmm

    rng = np.random.default_rng(T * D)
    pages = -(-T // P) + 2
    ld = H * D + pad
    x = {}
    for name in "kv":
        a = rng.standard_normal((T, ld)).astype(np.float32) * np.exp2(rng.integers(-8, 8, (T, 1))).astype(np.float32)
        a[rng.random((T, ld)) < 0.05] = 0
        x[name] = device(torch, a).to(dtypes(torch)[dtype])
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    if T > 3:
        slots[1], slots[3] = -1, pages * P            # neither is written
    before = rng.integers(0, 256, (2, pages, H, P * plain.token_bytes(type_, D)), dtype=np.uint8)
    kc, vc = device(torch, before[0]), device(torch, before[1])
    assert kc[0].numel() == qmm.cache_page_size(type_, H, D, P)
    qmm.qmm_cache_write(type_, dtype, x["k"], x["v"], ld, ld, T, H, D, device(torch, slots), kc, vc, pages, P)
    for name, cache, old in (("k", kc, before[0]), ("v", vc, before[1])):
        codes, scales = plain.cache_views(old, type_, H, D, P)
        codes, bits = codes.copy(), scales.view(np.uint16).copy()
        c, s = plain.block_quantize(type_, x[name].float().cpu().numpy()[:, : H * D].reshape(T, H, D))
        for i, slot in enumerate(slots):
            if 0 <= slot < pages * P:
                codes[slot // P, :, slot % P], bits[slot // P, :, slot % P] = c[i], s.view(np.uint16)[i]
        want = plain.make_chunks(type_, codes, bits.view(np.float16))
        np.testing.assert_array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
def test_write_special_values(torch, type_):
    import block_quantized_matmul_gb300 as qmm

    T, H, D, P = 10, 1, 64, 16
    f = np.float32
    x = np.random.default_rng(0).standard_normal((T, D)).astype(f)
    x[1] = 0
    x[2, :32] = np.where(np.arange(32) % 2, 2.0, -2.0)          # magnitudes tie: the first one's sign counts
    x[3, :32] = np.where(np.arange(32) % 2, -2.0, 2.0)
    x[3, :5] = 0.5
    x[4, 7], x[5, 40], x[6, 1] = np.nan, np.inf, -np.inf
    x[7, 3] = 1e7                                                 # scale beyond fp16 for either type
    x[8, :4] = [1e-42, -1e-41, 3e-44, 0]                          # scales that round to zero in fp16
    x[8, 4:] = 0
    x[9] = np.linspace(-127, 127, 64)
    caches = [torch.zeros(1, H, P * plain.token_bytes(type_, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    xd = device(torch, x)
    qmm.qmm_cache_write(type_, "f32", xd, xd, D, D, T, H, D, torch.arange(T, device="cuda"), caches[0], caches[1], 1, P)
    c, s = plain.block_quantize(type_, x.reshape(T, H, D))
    codes, scales = plain.cache_views(caches[0].cpu().numpy(), type_, H, D, P)
    np.testing.assert_array_equal(codes[0, 0, :T], c[:, 0])
    np.testing.assert_array_equal(np.isnan(scales[0, 0, :T]), np.isnan(s[:, 0]))
    np.testing.assert_array_equal(np.nan_to_num(scales[0, 0, :T]), np.nan_to_num(s[:, 0]))
    assert torch.equal(caches[0], caches[1])
    y = torch.empty(T, D, device="cuda")
    table, starts = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    qmm.qmm_cache_read(type_, caches[0], caches[1], 1, P, H, D, table, 1, starts, 1, T, "f32", y, None, D, 0)
    want = plain.block_values(type_, c, s)[:, 0].astype(f)
    np.testing.assert_array_equal(y.cpu().numpy(), want)
    assert np.isnan(want[[4, 6], :32]).all() and np.isnan(want[5, 32:]).all() and np.isnan(want[7, :32]).all()


class Case:
    """A cache full of random codes (some scales of free tokens NaN), a page table and ragged lengths."""

    def __init__(self, torch, type_, lens, H, D, P, seed=0, key_scale=0.1):
        rng = np.random.default_rng(seed)
        self.torch, self.type, self.lens, self.H, self.D, self.P = torch, type_, lens, H, D, P
        most = max(1, max(-(-n // P) for n in lens)) + 1
        self.n_pages = len(lens) * most + 2
        self.table = rng.permutation(self.n_pages)[: len(lens) * most].reshape(len(lens), most).astype(np.int32)
        self.codes, self.scales = {}, {}
        for name in "kv":
            hi = 256
            self.codes[name] = rng.integers(0, hi, (self.n_pages, H, P, plain.code_bytes(type_, D)), dtype=np.uint8)
            unit = (1 / 127 if type_ == "q8_0" else 1 / 8) * (key_scale if name == "k" else 1.0)
            s = unit * rng.uniform(0.2, 2.0, (self.n_pages, H, P, D // 32)) * rng.choice([-1, 1], (self.n_pages, H, P, D // 32))
            self.scales[name] = s.astype(np.float16)
        # what lies past a sequence's end, or in a free page, is not read: NaN and infinities there
        used = np.zeros((self.n_pages, P), bool)
        for s, n in enumerate(lens):
            pos = np.arange(n)
            used[self.table[s, pos // P], pos % P] = True
        for name in "kv":
            sc = np.moveaxis(self.scales[name], 2, 1)            # [pages, P, H, D/32]
            sc[~used] = np.nan
            self.scales[name] = np.ascontiguousarray(np.moveaxis(sc, 1, 2))

    def upload(self):
        t = self.torch
        self.k_cache = device(t, plain.make_chunks(self.type, self.codes["k"], self.scales["k"]))
        self.v_cache = device(t, plain.make_chunks(self.type, self.codes["v"], self.scales["v"]))
        self.pages = device(t, self.table)
        return self

    def dense(self, name, s):
        """fp64 [n, H, D] of sequence s."""
        pos = np.arange(self.lens[s])
        page, off = self.table[s, pos // self.P], pos % self.P
        return plain.block_values(self.type, self.codes[name][page, :, off], self.scales[name][page, :, off])


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,H,D,P,pad", [([1], 1, 32, 16, 0), ([0, 17, 0, 64, 65, 1, 0], 2, 64, 16, 0), ([300, 5], 3, 96, 128, 1),
                                            ([40, 0], 1, 256, 32, 8)])
def test_read(torch, type_, dtype, lens, H, D, P, pad):
    import block_quantized_matmul_gb300 as qmm

    c = Case(torch, type_, lens, H, D, P).upload()
    T, ld = sum(lens), H * D + pad
    starts = device(torch, np.concatenate(([0], np.cumsum(lens))).astype(np.int32))
    out = {n: torch.full((T, ld), -7.0, dtype=dtypes(torch)[dtype], device="cuda") for n in "kv"}
    qmm.qmm_cache_read(type_, c.k_cache, c.v_cache, c.n_pages, P, H, D, c.pages, c.table.shape[1], starts, len(lens), T, dtype,
                       out["k"], out["v"], ld, ld)
    for name in "kv":
        want = np.concatenate([c.dense(name, s).reshape(-1, H * D) for s in range(len(lens))])
        want = torch.from_numpy(want.astype(np.float32)).to(dtypes(torch)[dtype])
        assert torch.equal(out[name][:, : H * D].cpu(), want)
        assert (out[name][:, H * D:] == -7).all()
    only = torch.empty(T, H * D, dtype=dtypes(torch)[dtype], device="cuda")
    qmm.qmm_cache_read(type_, c.k_cache, c.v_cache, c.n_pages, P, H, D, c.pages, c.table.shape[1], starts, len(lens), T, dtype,
                       None, only, 0, H * D)
    assert torch.equal(only, out["v"][:, : H * D])


def test_read_pages_out_of_the_pool(torch):
    import block_quantized_matmul_gb300 as qmm

    c = Case(torch, "q8_0", [40, 40], 1, 64, 16)
    c.table[0, 1], c.table[1, 0] = -1, c.n_pages
    c.upload()
    starts = device(torch, np.array([0, 40, 80], np.int32))
    k = torch.full((80, 64), -7.0, device="cuda")
    qmm.qmm_cache_read("q8_0", c.k_cache, c.v_cache, c.n_pages, 16, 1, 64, c.pages, c.table.shape[1], starts, 2, 80, "f32", k, None, 64, 0)
    k = k.cpu().numpy()
    assert (k[16:32] == 0).all() and (k[40:56] == 0).all() and (k[:16] != 0).any() and (k[32:40] != 0).any() and (k[56:] != 0).any()


def run_attend(c, q, q_starts, lens, dtype, tree, scale, workspace=None, lse=True, ldq=None, stream=None, max_new=None, max_len=None):
    import block_quantized_matmul_gb300 as qmm

    torch = c.torch
    T, Hq, D = q.shape
    ldq = Hq * D if ldq is None else ldq
    qb = torch.full((T, ldq), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    qb[:, : Hq * D] = device(torch, q.reshape(T, -1)).to(dtypes(torch)[dtype])
    ob = torch.full((T, ldq), -7.0, dtype=dtypes(torch)[dtype], device="cuda")
    lb = torch.full((T, Hq), -7.0, device="cuda") if lse else None
    news = np.diff(q_starts)
    max_new = int(news.max()) if max_new is None else max_new
    max_len = int(max(lens)) if max_len is None else max_len
    if workspace is None:
        workspace = qmm.cache_attend_workspace_size(len(lens), max_new, c.H, Hq, D, max_len)
    ws = torch.full((workspace,), 0xFF, dtype=torch.uint8, device="cuda") if workspace else None
    td = device(torch, tree.astype(np.uint64).view(np.int64)) if tree is not None else None
    qmm.qmm_cache_attend(c.type, c.k_cache, c.v_cache, c.n_pages, c.P, c.H, D, c.pages, c.table.shape[1],
                         device(torch, q_starts.astype(np.int32)), device(torch, np.array(lens, np.int32)), len(lens), dtype, qb, ldq, T,
                         Hq, td, scale, max_new, max_len, ob, ldq, lb, ws, workspace, stream=stream)
    torch.cuda.synchronize()
    assert (ob[:, Hq * D:] == -7).all()
    return ob[:, : Hq * D].float().cpu().numpy().reshape(T, Hq, D), None if lb is None else lb.cpu().numpy(), \
        qb[:, : Hq * D].float().cpu().numpy().reshape(T, Hq, D)


def visible(n, new, tree, base):
    """bool [new, n] for new tokens whose tree words start at tree[base]."""
    seen = np.zeros((new, n), bool)
    first = n - new
    for i in range(new):
        for j in range(n):
            b = j - first
            seen[i, j] = b < 0 or (b <= i if tree is None else b < 64 and bool(int(tree[base + i]) >> b & 1))
    return seen


def check_attend(c, got, lse, q, q_starts, lens, tree, scale, dtype):
    Hq = q.shape[1]
    G = Hq // c.H
    for s, n in enumerate(lens):
        new = int(q_starts[s + 1] - q_starts[s])
        if new == 0:
            continue
        base = int(q_starts[s])
        seen = visible(n, new, tree, base)
        k, v = c.dense("k", s), c.dense("v", s)
        for hq in range(Hq):
            out, mag, ls, big = plain.attend(q[base:base + new, hq].astype(np.float64), k[:, hq // G], v[:, hq // G], seen, scale)
            # four roundings of 2^-11 (probabilities, values, two halves of slack), the fp32 scores, the output's rounding
            ds = 2.0 ** -20 * big[:, None]
            tol = (2.0 ** -9 + ds) * mag + plain.ULP[dtype] * np.abs(out) + 1e-6
            g = got[base:base + new, hq]
            np.testing.assert_array_equal(np.isnan(g), np.isnan(out))
            err = np.abs(np.nan_to_num(g) - np.nan_to_num(out))
            assert (err <= np.nan_to_num(tol, nan=1e9)).all(), (s, hq, float(err.max()), float(np.nanmin(tol)))
            if lse is not None:
                l = lse[base:base + new, hq]
                np.testing.assert_array_equal(np.isinf(l), np.isinf(ls))
                fine = np.isfinite(ls)
                assert (np.abs(l[fine] - ls[fine]) <= 1e-5 + 2.0 ** -20 * big[fine]).all()


def random_tree(rng, news):
    words = []
    for new in news:
        bits = []
        for i in range(new):
            up = rng.integers(-1, i) if i else -1
            bits.append((1 << i) | (bits[up] if up >= 0 else 0))
        words += bits
    return np.array(words, dtype=np.uint64)


ATTEND = [
    # lens, news, H, G, D, P
    ([1], [1], 1, 1, 64, 16),
    ([17], [1], 2, 4, 128, 16),
    ([0, 1, 15, 16, 17, 63, 64, 65, 130], [0, 1, 1, 1, 1, 1, 1, 1, 1], 2, 4, 64, 64),
    ([300, 5, 77], [1, 1, 1], 1, 8, 128, 32),
    ([260], [1], 1, 16, 96, 256),
    ([200, 33], [1, 1], 2, 3, 256, 128),
    ([50, 64], [1, 1], 1, 7, 32, 16),
    ([100, 90], [1, 1], 1, 2, 160, 32),
    ([100, 90], [1, 1], 1, 1, 192, 64),
    ([70, 20], [1, 2], 1, 64, 128, 16),
    ([129, 4, 70], [5, 4, 16], 2, 4, 128, 64),
    ([200, 64, 65, 40], [64, 64, 1, 33], 1, 4, 64, 16),
    ([150], [64], 1, 1, 256, 32),
    ([90, 100], [20, 17], 2, 5, 96, 128),
    ([2500, 700], [1, 3], 2, 4, 128, 64),
]


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("lens,news,H,G,D,P", ATTEND)
def test_attend(torch, type_, dtype, tree, lens, news, H, G, D, P):
    rng = np.random.default_rng(D + len(lens))
    c = Case(torch, type_, lens, H, D, P, seed=D).upload()
    q_starts = np.concatenate(([0], np.cumsum(news)))
    words = random_tree(rng, news) if tree else None
    q = rng.standard_normal((q_starts[-1], H * G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, dtype, words, 1 / math.sqrt(D))
    check_attend(c, got, lse, q, q_starts, lens, words, 1 / math.sqrt(D), dtype)


def test_attend_chain_longer_than_64(torch):
    lens, news = [300, 150], [150, 150]
    c = Case(torch, "q8_0", lens, 1, 64, 32).upload()
    q = np.random.default_rng(1).standard_normal((300, 3, 64)).astype(np.float32)
    q_starts = np.array([0, 150, 300])
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.125)
    check_attend(c, got, lse, q, q_starts, lens, None, 0.125, "bf16")


@pytest.mark.parametrize("workspace", [0, None, 64 << 20])
@pytest.mark.parametrize("news", [[1, 1], [6, 3]])
def test_attend_long_sequences_split_or_not(torch, news, workspace):
    lens = [20011, 4096]
    c = Case(torch, "q8_0", lens, 1, 128, 64).upload()
    q_starts = np.concatenate(([0], np.cumsum(news)))
    q = 3 * np.random.default_rng(2).standard_normal((q_starts[-1], 4, 128)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "f16", None, 0.3, workspace=workspace)
    check_attend(c, got, lse, q, q_starts, lens, None, 0.3, "f16")
    # the same bits again, and without the log-sums
    again, _, _ = run_attend(c, q, q_starts, lens, "f16", None, 0.3, workspace=workspace, lse=False)
    np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("new", [1, 9])
def test_attend_rows_that_see_nothing(torch, new):
    """No context and an empty tree word: the row is 0 and its log-sum -inf; others of the sequence are not touched."""
    lens, news = [new, 40, 0], [new, new, 0]
    c = Case(torch, "q8_0", lens, 2, 64, 16).upload()
    q_starts = np.array([0, new, 2 * new, 2 * new])
    tree = random_tree(np.random.default_rng(3), news)
    tree[new - 1] = 0                      # sequence 0 has no context
    tree[new] = 0                          # sequence 1 has: the row sees the context alone
    q = np.random.default_rng(4).standard_normal((2 * new, 4, 64)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", tree, 0.125)
    assert (got[new - 1] == 0).all() and np.isneginf(lse[new - 1]).all()
    check_attend(c, got, lse, q, q_starts, lens, tree, 0.125, "bf16")


def test_attend_nan_and_infinity_reach_only_who_sees_them(torch):
    lens, news = [60, 200], [8, 8]
    c = Case(torch, "q8_0", lens, 1, 128, 16)
    q_starts = np.array([0, 8, 16])
    tree = np.array([1 << i for i in range(8)] * 2, dtype=np.uint64)     # each new token sees itself and the context
    for s, n in enumerate(lens):
        for b, name, block in ((2, "v", 1), (5, "k", 3), (6, "v", 0)):
            pos = n - 8 + b
            c.scales[name][c.table[s, pos // 16], 0, pos % 16, block] = np.nan if b != 6 else np.inf
            c.codes[name][c.table[s, pos // 16], 0, pos % 16, 32 * block:32 * block + 32] |= 1    # (no 0 * inf)
    c.upload()
    q = np.random.default_rng(5).standard_normal((16, 2, 128)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", tree, 0.1)
    for base in (0, 8):
        bad = ~np.isfinite(got[base:base + 8])
        assert bad[2, :, 32:64].all() and bad[5].all() and bad[6, :, :32].all()
        assert bad.sum() == 2 * (32 + 128 + 32)
    for name in "kv":                      # the same without them, for the other rows
        c.scales[name] = np.where(np.isfinite(c.scales[name]), c.scales[name], np.float16(0.01))
    clean, _, _ = run_attend(c.upload(), q, q_starts, lens, "bf16", tree, 0.1)
    for base in (0, 8):
        for i in (0, 1, 3, 4, 7):
            np.testing.assert_array_equal(got[base + i], clean[base + i])


def test_attend_large_scores_and_small_values(torch):
    """Scores in the hundreds (one key dominates), values around 1e-4, queries of mixed size."""
    lens = [500]
    c = Case(torch, "q8_0", lens, 1, 64, 64, key_scale=8.0)
    c.scales["v"] = (c.scales["v"].astype(np.float32) * 1e-4).astype(np.float16)
    c.upload()
    q = np.random.default_rng(6).standard_normal((1, 4, 64)).astype(np.float32) * np.array([1e-3, 1, 30, 1e3], np.float32)[None, :, None]
    got, lse, q = run_attend(c, q, np.array([0, 1]), lens, "bf16", None, 0.125)
    Hq = 4
    k, v = c.dense("k", 0)[:, 0], c.dense("v", 0)[:, 0]
    for hq in range(Hq):
        out, mag, ls, big = plain.attend(q[:, hq].astype(np.float64), k, v, np.ones((1, 500), bool), 0.125)
        tol = (2.0 ** -9 + 2.0 ** -20 * big[:, None]) * mag + 2.0 ** -8 * np.abs(out) + 1e-9
        assert (np.abs(got[:, hq] - out) <= tol).all(), hq


def test_attend_pages_out_of_the_pool_are_not_seen(torch):
    lens = [64, 40]
    c = Case(torch, "q4_0", lens, 1, 64, 16).upload()
    q = np.random.default_rng(7).standard_normal((2, 2, 64)).astype(np.float32)
    table = c.table.copy()
    c.table[0, 1], c.table[1, 0] = -1, c.n_pages + 5
    c.pages = device(torch, c.table)
    got, lse, q = run_attend(c, q, np.array([0, 1, 2]), lens, "f16", None, 0.125)
    c.table = table
    for s, hide in ((0, slice(16, 32)), (1, slice(0, 16))):
        seen = np.ones((1, lens[s]), bool)
        seen[:, hide] = False
        for hq in range(2):
            out, mag, ls, _ = plain.attend(q[s:s + 1, hq].astype(np.float64), c.dense("k", s)[:, 0], c.dense("v", s)[:, 0], seen, 0.125)
            assert (np.abs(got[s, hq] - out[0]) <= 2.0 ** -8 * mag[0] + 1e-6).all()
            assert abs(lse[s, hq] - ls[0]) < 1e-4


def test_attend_strided_rows_on_another_stream(torch):
    lens, news = [700, 40, 333], [1, 4, 2]
    c = Case(torch, "q8_0", lens, 2, 128, 64).upload()
    q_starts = np.array([0, 1, 5, 7])
    q = np.random.default_rng(8).standard_normal((7, 8, 128)).astype(np.float32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.088, ldq=8 * 128 + 24, stream=s)
    check_attend(c, got, lse, q, q_starts, lens, None, 0.088, "bf16")


def test_hints_larger_than_needed(torch):
    lens, news = [70, 9], [2, 1]
    c = Case(torch, "q8_0", lens, 1, 64, 16).upload()
    q = np.random.default_rng(9).standard_normal((3, 4, 64)).astype(np.float32)
    got, lse, q = run_attend(c, q, np.array([0, 2, 3]), lens, "f16", None, 0.125, max_new=40, max_len=100000)
    check_attend(c, got, lse, q, np.array([0, 2, 3]), lens, None, 0.125, "f16")


def test_offsets_past_32_bits(torch):
    """A pool of more than 2^32 bytes: the last pages are written, read and attended at their own place."""
    import block_quantized_matmul_gb300 as qmm

    H, D, P = 8, 128, 64
    size = qmm.cache_page_size("q8_0", H, D, P)
    n_pages = (1 << 32) // size + 40
    kc, vc = (torch.zeros(n_pages * size, dtype=torch.uint8, device="cuda") for _ in range(2))
    T = 100
    rng = np.random.default_rng(10)
    k, v = (device(torch, rng.standard_normal((T, H * D)).astype(np.float32)) for _ in range(2))
    table = np.array([[n_pages - 1, n_pages - 7]], np.int32)
    pos = np.arange(T)
    slots = device(torch, table[0, pos // P].astype(np.int64) * P + pos % P)
    qmm.qmm_cache_write("q8_0", "f32", k, v, H * D, H * D, T, H, D, slots, kc, vc, n_pages, P)
    out = torch.empty(T, H * D, device="cuda")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    pages = device(torch, table)
    qmm.qmm_cache_read("q8_0", kc, vc, n_pages, P, H, D, pages, 2, starts, 1, T, "f32", out, None, H * D, 0)
    c, s = plain.block_quantize("q8_0", k.cpu().numpy().reshape(T, H, D))
    kd = plain.block_values("q8_0", c, s)
    np.testing.assert_array_equal(out.cpu().numpy().reshape(T, H, D), kd.astype(np.float32))
    assert int(kc[: (n_pages - 8) * size].any()) == 0
    q = device(torch, rng.standard_normal((1, H * D)).astype(np.float32)).to(torch.bfloat16)
    o = torch.empty_like(q)
    qmm.qmm_cache_attend("q8_0", kc, vc, n_pages, P, H, D, pages, 2, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                         starts[1:].contiguous(), 1, "bf16", q, H * D, 1, H, None, 0.088, 1, T, o, H * D, None, None, 0)
    c, s = plain.block_quantize("q8_0", v.cpu().numpy().reshape(T, H, D))
    vd = plain.block_values("q8_0", c, s)
    qf = q.float().cpu().numpy().reshape(H, D).astype(np.float64)
    for h in range(H):
        want, mag, _, _ = plain.attend(qf[h:h + 1], kd[:, h], vd[:, h], np.ones((1, T), bool), 0.088)
        got = o.float().cpu().numpy().reshape(H, D)[h]
        assert (np.abs(got - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -8 * mag[0]).all()
