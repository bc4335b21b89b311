"""Attention over the block-quantized cache in batches with empty sequences (slots of a padded batch) that are split:
every piece of every sequence belongs to a CTA.  Tolerances are those of test_gpu_cache.check_attend; workspaces are
filled with NaN and outputs preset, so that a piece nobody computes shows."""
import math

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


BATCHES = [
    # lens, new tokens a sequence, H, G, D, P, max_len: their steps of 128 keys fit one wave of CTAs, with the empty ones they do not
    ([433, 0, 1904], 1, 16, 2, 64, 64, 4096),
    ([0, 500] * 8, 1, 8, 4, 64, 64, 4096),
    ([0, 512, 512, 1024] + [256] * 11, 1, 8, 1, 128, 16, 4096),       # empty at the start
    ([0] * 9 + [384] * 2 + [512] * 8, 1, 8, 2, 64, 64, 4096),
    ([512] * 8 + [384] * 2 + [0] * 9, 1, 8, 2, 64, 64, 4096),         # at the end
    ([0, 512] * 8 + [0] * 24, 1, 4, 8, 32, 32, 4096),                 # more than a warp has lanes
    ([60, 498, 0], 20, 8, 16, 64, 64, 498),                           # 320 rows, on tcgen05
    ([135, 0, 0, 262, 0, 0, 1229, 154], 9, 16, 4, 32, 64, 1229),      # two waves
    ([0] * 12, 1, 2, 4, 64, 16, 1000),                                # nothing but empty ones
]


@pytest.mark.parametrize("type_,dtype", [("q8_0", "bf16"), ("q4_0", "f16")])
@pytest.mark.parametrize("padded,lens,new,H,G,D,P,max_len", [(p, *b) for b in BATCHES for p in (False, True) if p or any(b[0])])
def test_every_piece_has_a_cta(torch, type_, dtype, padded, lens, new, H, G, D, P, max_len):
    """`padded`: the empty sequences have rows of q too, which come out as 0 with a log-sum of -inf."""
    news = [new if n or padded else 0 for n in lens]
    q_starts = np.concatenate(([0], np.cumsum(news)))
    c = Case(torch, type_, lens, H, D, P, seed=len(lens)).upload()
    q = np.random.default_rng(2).standard_normal((int(q_starts[-1]), H * G, D)).astype(np.float32)
    got, lse, q = run_attend(c, q, q_starts, lens, dtype, None, 1 / math.sqrt(D), max_len=max_len)
    for s, n in enumerate(lens):
        if n == 0:
            rows = slice(q_starts[s], q_starts[s + 1])
            assert (got[rows] == 0).all() and np.isneginf(lse[rows]).all()
    keep = [s for s, n in enumerate(lens) if n]
    for s in keep:
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__, table=c.table[s:s + 1], lens=[lens[s]])
        rows = slice(q_starts[s], q_starts[s + 1])
        check_attend(one, got[rows], lse[rows], q[rows], np.array([0, news[s]]), [lens[s]], None, 1 / math.sqrt(D), dtype)
