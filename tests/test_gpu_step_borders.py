"""The calls of a decode step at the borders of what their arguments promise: sequences as long as max_len's last page and one
token longer."""
import numpy as np
import pytest

from tests.test_gpu_cache import Case
from tests.test_gpu_sparse import gpu_bounds, gpu_select, plain_choice, torch  # noqa: F401 (a fixture)

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
