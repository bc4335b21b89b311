"""Attention over the block-quantized cache: rows of sequences that do not lie in q, and rows of no sequence, are left
as they are, whether their sequence would be split or not."""
import numpy as np
import pytest

from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, check_attend, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


@pytest.mark.parametrize("new,G", [(1, 4), (12, 4), (12, 1)])
@pytest.mark.parametrize("workspace", [0, None], ids=["whole", "split"])
@pytest.mark.parametrize("case", ["past_the_end", "behind_the_last", "before_the_first", "one_sequence"])
def test_rows_that_are_not_computed_keep_what_they_hold(torch, case, new, G, workspace):
    lens = [700, 900]
    if case == "past_the_end":                                 # the second sequence starts in q and ends past it
        q_starts, rows = np.array([0, new, 3 * new]), 2 * new
    elif case == "behind_the_last":                            # the last rows of q belong to nobody
        q_starts, rows = np.array([0, new, 2 * new]), 3 * new
    elif case == "before_the_first":                           # the first sequence starts before q: only the second lies in it
        q_starts, rows = np.array([-new, new, 2 * new]), 2 * new
    else:
        lens, q_starts, rows = [900], np.array([0, 2 * new]), new
    c = Case(torch, "q8_0", lens, 1, 64, 16).upload()
    q = np.random.default_rng(2).standard_normal((rows, G, 64)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.1, workspace=workspace, max_new=2 * new)
    left = np.ones(rows, bool)
    for s, n in enumerate(lens):
        a, b = q_starts[s], q_starts[s + 1]
        if a < 0 or b > rows:
            continue
        left[a:b] = False
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__, table=c.table[s:s + 1], lens=[n])
        check_attend(one, got[a:b], lse[a:b], q[a:b], np.array([0, b - a]), [n], None, 0.1, "bf16")
    assert (got[left] == -7).all() and (lse[left] == -7).all()
