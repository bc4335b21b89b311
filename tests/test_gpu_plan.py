"""The plan of a step on the GPU against its plain form: every output, whole."""
import numpy as np
import pytest

from tests import plain_step as step
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


def make(rng, lens, news, P, ld=None, free=None, extra=3):
    """Page tables with distinct pages, the rest of them free in a ring that has gone round."""
    held = [step.up(min(max(n, 0), (ld or 1 << 30) * P), P) for n in lens]
    need = [step.up(n + m, P) - h if m > 0 else 0 for n, m, h in zip(lens, news, held)]
    ld = ld or max(1, max(h + k for h, k in zip(held, need)))
    free = sum(need) + extra if free is None else free
    total = sum(held) + free
    order = rng.permutation(total + 5)
    pages = np.full((len(lens), ld), -9, np.int32)
    at = 0
    for s, h in enumerate(held):
        pages[s, : min(h, ld)] = order[at : at + min(h, ld)]
        at += h
    n_ring = max(1, total)
    first = int(rng.integers(0, 5 * n_ring))
    ring = np.full(n_ring, -5, np.int32)
    for i in range(free):
        ring[(first + i) % n_ring] = order[at + i]
    return pages, ring, np.array([first, first + free], np.int64)


def run(torch, lens, news, P, pages, ring, ring_at, T, alias=False, positions=True, stream=None):
    import block_quantized_matmul_gb300 as qmm

    d = lambda a, t: torch.from_numpy(np.array(a, dtype=t)).cuda()  # noqa: E731
    n = len(lens)
    out = {"lens": d(lens, np.int32), "news": d(news, np.int32), "pages": d(pages, np.int32), "ring": d(ring, np.int32), "ring_at": d(ring_at, np.int64),
           "q_starts": d([-7] * (n + 2), np.int32), "kv_lens": d([-7] * n, np.int32), "slots": d([-7] * (T + 1), np.int64),
           "positions": d([-7] * (T + 1), np.int32) if positions else None}
    out["next_lens"] = out["lens"] if alias else d([-7] * n, np.int32)
    out["next_at"] = out["ring_at"] if alias else d([-7] * 2, np.int64)
    qmm.qmm_cache_plan(out["lens"], out["news"], n, P, out["pages"], pages.shape[1], out["ring"], len(ring), out["ring_at"], T, out["q_starts"],
                       out["kv_lens"], out["slots"], out["positions"], out["next_lens"], out["next_at"], stream=stream)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out.items() if v is not None}
    assert got["q_starts"][-1] == -7 and got["slots"][-1] == -7                     # nothing behind the end
    got["q_starts"], got["slots"] = got["q_starts"][:-1], got["slots"][:-1]
    if positions:
        assert got["positions"][-1] == -7
        got["positions"] = got["positions"][:-1]
    return got


def check(got, want):
    for name, w in want.items():
        if name in got:
            np.testing.assert_array_equal(got[name], w, err_msg=name)


CASES = [
    # lens, news, P, T - rows
    ([0], [1], 16, 0), ([16], [1], 16, 0), ([15], [1], 16, 2), ([5], [0], 16, 0), ([40], [-1], 16, 0), ([0], [-1], 16, 1),
    ([0, 3, 16, 17, 0], [1, 0, 1, -1, 40], 16, 3), ([100, 64, 63, 0], [64, 1, 2, 300], 64, 0), ([255, 256, 257, 1], [1, 1, -2, 513], 256, 5),
]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("lens,news,P,more", CASES)
def test_plan(torch, lens, news, P, more, alias):
    pages, ring, at = make(np.random.default_rng(len(lens)), lens, news, P)
    T = sum(max(0, m) for m in news) + more
    check(run(torch, lens, news, P, pages, ring, at, T, alias), step.plan(lens, news, P, pages, ring, at, T))


@pytest.mark.parametrize("n_seq,top,new,P", [(31, 100, 1, 16), (256, 500, 4, 32), (257, 500, 4, 16), (1024, 3000, 2, 64), (1025, 300, 1, 16),
                                             (3000, 200, 9, 128), (40, 2000, 3000, 16), (700, 100, 300, 256)])
@pytest.mark.parametrize("share", [1.0, 0.5, 0.0])
def test_plan_of_many(torch, n_seq, top, new, P, share):
    """Idle, finished and waiting requests among running ones; the ring holds a share of what is wanted."""
    rng = np.random.default_rng(n_seq + int(10 * share))
    lens = rng.integers(0, top, n_seq)
    news = np.where(rng.random(n_seq) < 0.1, -1, rng.integers(0, new + 1, n_seq))
    want = sum(step.up(int(n + m), P) - step.up(int(n), P) for n, m in zip(lens, news) if m > 0)
    pages, ring, at = make(rng, lens.tolist(), news.tolist(), P, free=int(want * share))
    T = int(np.maximum(news, 0).sum()) + 7
    alias = n_seq % 2 == 1
    check(run(torch, lens, news, P, pages, ring, at, T, alias, positions=share > 0), step.plan(lens, news, P, pages, ring, at, T))


def test_rows_past_t_and_tables_that_are_full(torch):
    """A sequence whose rows pass T waits, and so do all behind it that have rows; one whose table is full waits alone."""
    lens, news, P = [10, 30, 0, 40, 5, 0], [4, 3, 0, 20, 1, 2], 16
    pages, ring, at = make(np.random.default_rng(5), lens, news, P, ld=3)
    for T in (0, 6, 7, 26, 27, 28, 30, 50):
        want = step.plan(lens, news, P, pages, ring, at, T)
        check(run(torch, lens, news, P, pages, ring, at, T), want)
    assert want["kv_lens"].tolist() == [14, 33, 0, 0, 6, 2]                         # 40 + 20 tokens do not fit 3 pages of 16


def test_lengths_out_of_range_count_as_the_nearest(torch):
    lens, news, P = [-5, 100, 1 << 30], [1, -1, 0], 16
    pages, ring, at = make(np.random.default_rng(6), lens, news, P, ld=2, free=1, extra=0)
    ring = np.concatenate((ring[:1] * 0 + 3, np.full(4, -5, np.int32)))
    at = np.array([10, 11])
    check(run(torch, lens, news, P, pages, ring, at, 1), step.plan(lens, news, P, pages, ring, at, 1))


def test_repeated_calls_and_other_streams_give_the_same(torch):
    lens, news, P = [3, 70, 0, 12], [5, 1, 100, -1], 32
    pages, ring, at = make(np.random.default_rng(7), lens, news, P)
    T = 106
    want = step.plan(lens, news, P, pages, ring, at, T)
    s = torch.cuda.Stream()
    check(run(torch, lens, news, P, pages, ring, at, T, stream=s), want)
    got = run(torch, lens, news, P, want["pages"], want["ring"], at, T)             # the state is as after one call
    check(got, want)


def test_a_captured_graph_carries_the_state(torch):
    """With lens and the ring's counters replaced in place, replays are steps: pages go round until none is free."""
    import block_quantized_matmul_gb300 as qmm

    rng = np.random.default_rng(8)
    n, P, steps = 5, 16, 60
    lens, news = np.array([0, 14, 15, 16, 31]), np.ones(5, int)
    pages, ring, at = make(rng, lens.tolist(), news.tolist(), P, ld=8, free=9)
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()  # noqa: E731
    L, W, G, R = i32(lens), i32(news), i32(pages), i32(ring)
    A = torch.from_numpy(at).cuda()
    qs, kv, slots = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), i32([0] * n), torch.zeros(n, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_cache_plan(L, W, n, P, G, 8, R, len(ring), A, n, qs, kv, slots, None, L, A)
    for i in range(steps):
        if i == 25:                                                                   # a request is done: its pages come back
            W[1] = -1
            news[1] = -1
        if i == 26:
            W[1] = 1
            news[1] = 1
        want = step.plan(lens, news, P, pages, ring, at, n)
        graph.replay()
        torch.cuda.synchronize()
        lens, pages, ring, at = want["next_lens"], want["pages"], want["ring"], want["next_at"]
        for name, t in (("q_starts", qs), ("kv_lens", kv), ("slots", slots), ("next_lens", L), ("pages", G), ("ring", R), ("next_at", A)):
            np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=f"{name} after step {i}")
    assert (want["kv_lens"] == 0).any()                                              # somebody waits at the end
