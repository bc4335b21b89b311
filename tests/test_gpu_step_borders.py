"""The calls of a decode step at the borders of what their arguments promise: sequences as long as max_len's last page and one
token longer, and sequences whose rows pass the step's."""
import numpy as np
import pytest

from tests import plain_step as step
from tests.test_gpu_cache import Case, run_attend
from tests.test_gpu_plan import check as check_plan, run as run_plan
from tests.test_gpu_sparse import gpu_attend, gpu_bounds, gpu_select, plain_choice, torch  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_len", [1, 100, 128, 129, 512, 513, 576])
@pytest.mark.parametrize("budget", [2, 20])
def test_max_len_counts_whole_pages(torch, max_len, budget):  # noqa: F811
    """Sequences in max_len's last page get their pages, those beyond it none, whether all pages are chosen or some."""
    P, lens = 64, [1, 64, 65, 100, 120, 128, 129, 500, 512, 513, 576]
    news = [1] * len(lens)
    c = Case(torch, "q8_0", lens, 2, 64, P, seed=50).upload()
    bounds = gpu_bounds(c, lens)
    q = np.random.default_rng(51).standard_normal((len(lens), 4, 64)).astype(np.float32)
    got, q = gpu_select(c, bounds, q, news, "bf16", None, 0, 1, budget, max_len=max_len)
    got, want = got.cpu().numpy(), plain_choice(c, bounds, q, news, False, 0, 1, budget)
    for i, n in enumerate(lens):
        fits = -(-n // P) <= -(-max_len // P)
        np.testing.assert_array_equal(got[i], want[i] if fits else np.full_like(want[i], -1), err_msg=str(n))


@pytest.mark.parametrize("T", [5, 6, 7, 9, 12])
@pytest.mark.parametrize("free", [0, 3])
def test_rows_of_sequences_that_wait(torch, T, free):  # noqa: F811
    """The plan's outputs into the calls that take them.  Rows of a sequence that waits for pages are 0; those of one whose rows pass T,
    and of all behind it, keep what the buffers held, below T too."""
    P, lens, news = 16, [32, 20, 16, 40], [2, 4, 3, 3]                        # rows 0, 2, 6, 9 to 12; the first and the third need a page
    after = [n + m for n, m in zip(lens, news)]
    c = Case(torch, "q8_0", after, 2, 64, P, seed=60).upload()
    old = [-(-n // P) for n in lens]
    table = np.array([[c.table[s, k] if k < old[s] else -1 for k in range(c.table.shape[1])] for s in range(4)], np.int32)
    wanted = [c.table[s, k] for s in range(4) for k in range(old[s], -(-after[s] // P))]
    ring = np.array(wanted[:free] + [-5] * (8 - min(free, len(wanted))), np.int32)
    at = np.array([0, min(free, len(wanted))])
    want = step.plan(lens, news, P, table, ring, at, T)
    got = run_plan(torch, lens, news, P, table, ring, at, T)
    check_plan(got, want)
    starts, kv = got["q_starts"], got["kv_lens"]
    assert starts.tolist() == [0, 2, 6, 9, 12] and (free == 3) == (kv[0] > 0) and kv[1] == (24 if T >= 6 else 0)
    c.table, c.pages = got["pages"], torch.from_numpy(got["pages"]).cuda()
    bounds = gpu_bounds(c, after)
    rng = np.random.default_rng(61)
    q = rng.standard_normal((T, 4, 64)).astype(np.float32)
    chosen, _ = gpu_select(c, bounds, q, news, "bf16", None, 0, 1, 8, max_new=4, lens=kv.tolist(), max_len=64)
    out, lse, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen, lens=kv.tolist())
    all_, lse2, qr = run_attend(c, q, starts, kv.tolist(), "bf16", None, 0.1, max_len=64)
    for s in range(4):
        a, b = starts[s], min(starts[s + 1], T)
        if starts[s + 1] > T:
            assert (chosen[a:b] == -7).all() and (out[a:b] == -7).all() and (lse[a:b] == -7).all() and (all_[a:b] == -7).all() and (lse2[a:b] == -7).all()
        elif kv[s] == 0:
            assert (chosen[a:b] == -1).all() and (out[a:b] == 0).all() and np.isneginf(lse[a:b]).all() and (all_[a:b] == 0).all()
        else:
            assert (out[a:b] != -7).all() and (np.abs(out[a:b] - all_[a:b]) <= 2.0 ** -7 * np.abs(all_).max()).all()


def test_a_sequence_without_rows_behind_the_steps_end_waits(torch):  # noqa: F811
    lens, news, P = [10, 20, 30, 40], [4, 9, 0, -1], 16
    table = np.arange(12, dtype=np.int32).reshape(4, 3)
    ring, at = np.full(8, 12, np.int32), np.array([0, 4])
    for T in (3, 4, 12, 13):
        got = run_plan(torch, lens, news, P, table, ring, at, T)
        check_plan(got, step.plan(lens, news, P, table, ring, at, T))
        assert got["kv_lens"].tolist() == [14 if T >= 4 else 0, 29 if T >= 13 else 0, 30 if T >= 13 else 0, 0]
        assert got["next_lens"].tolist() == [14 if T >= 4 else 10, 29 if T >= 13 else 20, 30, 0]
