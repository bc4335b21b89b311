"""Attention over the block-quantized cache where sequences are split among CTAs: many of them, uneven ones, whole
batches that need no split, and lengths that change under a captured graph.  The tolerances are those of
test_gpu_cache.check_attend."""
import math

import numpy as np
import pytest

from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, check_attend, device, random_tree, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


def spread(n, lo, hi):
    return [int(x) for x in np.random.default_rng(n).permutation(np.linspace(lo, hi, n).astype(int))]


SPLITS = [
    # lens, new tokens a sequence, H, G, D, P
    (spread(40, 0, 700), 1, 1, 8, 64, 16),                     # more sequences than a warp has lanes
    (spread(100, 1, 400), 1, 2, 2, 32, 32),                    # over half the GPU's places: one wave or two
    ([128, 256, 384, 129, 257, 127], 1, 2, 4, 64, 64),         # at, before and past whole steps
    ([3000] + [1] * 20, 1, 2, 3, 128, 64),                     # one sequence is nearly all
    ([1, 0, 2600, 0], 1, 1, 1, 256, 16),
    ([900, 30, 400], 4, 2, 4, 96, 16),                         # 16 rows
    ([900, 30, 400, 31], 8, 1, 4, 128, 32),                    # 32 rows
    ([1500, 40, 400], 20, 1, 4, 64, 16),                       # 80 rows, on tcgen05
    (spread(12, 60, 500), 9, 8, 4, 32, 64),                    # the same over half its places
    ([1030, 200], 20, 1, 16, 128, 64),                         # 320 rows: three tiles of them
]


@pytest.mark.parametrize("type_,dtype", [("q8_0", "f16"), ("q4_0", "bf16")])
@pytest.mark.parametrize("lens,new,H,G,D,P", SPLITS)
def test_splits(torch, type_, dtype, lens, new, H, G, D, P):
    news = [min(new, n) for n in lens]
    q_starts = np.concatenate(([0], np.cumsum(news)))
    c = Case(torch, type_, lens, H, D, P, seed=len(lens)).upload()
    tree = random_tree(np.random.default_rng(1), news) if new > 4 else None
    q = np.random.default_rng(2).standard_normal((int(q_starts[-1]), H * G, D)).astype(np.float32)
    scale = 1 / math.sqrt(D)
    got, lse, rounded = run_attend(c, q, q_starts, lens, dtype, tree, scale)
    check_attend(c, got, lse, rounded, q_starts, lens, tree, scale, dtype)
    again, lse2, _ = run_attend(c, q, q_starts, lens, dtype, tree, scale)
    np.testing.assert_array_equal(got, again)
    np.testing.assert_array_equal(lse, lse2)


@pytest.mark.parametrize("new,G,D", [(1, 8, 128), (20, 4, 64)])
@pytest.mark.parametrize("max_len", [100000, 1])
def test_max_len_only_bounds_the_splits(torch, new, G, D, max_len):
    """A bound far above the lengths (nothing is split) or below them changes no result beyond rounding."""
    lens = [100, 60, 300]
    q_starts = np.arange(4) * new
    c = Case(torch, "q8_0", lens, 1, D, 16).upload()
    q = np.random.default_rng(2).standard_normal((3 * new, G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.1, max_len=max_len)
    check_attend(c, got, lse, q, q_starts, lens, None, 0.1, "bf16")


@pytest.mark.parametrize("splits", [2, 3])
def test_small_workspace_splits_less(torch, splits):
    import block_quantized_matmul_gb300 as qmm

    lens, G, D = [2000, 500], 4, 64
    c = Case(torch, "q8_0", lens, 1, D, 16).upload()
    q = np.random.default_rng(2).standard_normal((2, G, D)).astype(np.float32)
    need = splits * -(-2 * G * (D + 2) * 4 // 256) * 256
    assert need < qmm.cache_attend_workspace_size(2, 1, 1, G, D, 2000)
    got, lse, q = run_attend(c, q, np.arange(3), lens, "f16", None, 0.1, workspace=need)
    check_attend(c, got, lse, q, np.arange(3), lens, None, 0.1, "f16")


@pytest.mark.parametrize("new,G", [(1, 4), (12, 4)])
@pytest.mark.parametrize("workspace", [0, None])
def test_rows_that_do_not_lie_in_q_are_skipped(torch, new, G, workspace):
    lens = [400, 700, 900]
    c = Case(torch, "q8_0", lens, 1, 64, 16).upload()
    q = np.random.default_rng(2).standard_normal((2 * new, G, 64)).astype(np.float32)
    q_starts = np.array([0, new, 2 * new, 3 * new])            # the third sequence's rows are past q's end
    got, lse, q = run_attend(c, q, q_starts, lens, "bf16", None, 0.1, workspace=workspace, max_new=new)
    check_attend(c, got, lse, q, q_starts[:3], lens[:2], None, 0.1, "bf16")


@pytest.mark.parametrize("new,G,D", [(1, 8, 128), (16, 4, 64)])
def test_lengths_change_under_a_graph(torch, new, G, D):
    """One captured call serves every set of lengths, and the calls after it see its results."""
    import block_quantized_matmul_gb300 as qmm

    most, sets = 2000, [[2000, 40, 700], [new, new, new], [300, 2000, 2000], [0, 129, 1500]]
    c = Case(torch, "q8_0", [most] * 3, 1, D, 16).upload()
    q_np = np.random.default_rng(2).standard_normal((3 * new, G, D)).astype(np.float32)
    q = device(torch, q_np.reshape(3 * new, -1)).to(torch.bfloat16)
    out, out2 = (torch.empty_like(q) for _ in range(2))
    lse = torch.empty(3 * new, G, device="cuda")
    starts, lens = device(torch, (np.arange(4) * new).astype(np.int32)), torch.zeros(3, dtype=torch.int32, device="cuda")
    need = qmm.cache_attend_workspace_size(3, new, 1, G, D, most)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(src, dst):
        qmm.qmm_cache_attend("q8_0", c.k_cache, c.v_cache, c.n_pages, 16, 1, D, c.pages, c.table.shape[1], starts, lens, 3, "bf16", src,
                             G * D, 3 * new, G, None, 0.1, new, most, dst, G * D, lse, ws, need)

    call(q, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, out)
        call(out, out2)                                        # reads what the call before it wrote
    for values in sets:
        values = [max(v, new) if v else 0 for v in values]
        lens.copy_(torch.tensor(values, dtype=torch.int32))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        c.lens = values
        for src, dst in ((q, out), (out, out2)):
            a = src.float().cpu().numpy().reshape(-1, G, D)
            b = dst.float().cpu().numpy().reshape(-1, G, D)
            keep = [s for s in range(3) if values[s] >= new]
            for s in range(3):
                if s not in keep:
                    assert (b[s * new:(s + 1) * new] == 0).all()
            for s in keep:
                one = Case.__new__(Case)
                one.__dict__.update(c.__dict__, table=c.table[s:s + 1], lens=[values[s]])
                check_attend(one, b[s * new:(s + 1) * new], None, a[s * new:(s + 1) * new], np.array([0, new]), [values[s]], None, 0.1, "bf16")
