"""How exact the attention over the block-quantized cache is for fp16 outputs, where the probabilities take part in two
terms: values whose scales are powers of two (so that they are exact in fp16) of both signs leave the output's own
rounding and the fp32 steps alone.

The bound: scores are sums of at most 256 fp32 products and sums, and the exponential is off by 2^-22; a relative error of
2^-20 * (largest sum of |scale * q k|) + 2^-20 in each probability covers both.  The two terms hold a probability to 2^-22;
one term alone, off by up to 2^-12, does not pass."""
import math

import numpy as np
import pytest

from tests import plain_ops as plain
from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
@pytest.mark.parametrize("lens,new,G,D", [([300, 40], 1, 4, 128), ([90, 700], 4, 4, 64), ([60, 500], 8, 4, 128), ([200, 333], 20, 4, 64),
                                          ([300], 1, 5, 256)])
def test_fp16_outputs_are_rounded_once(torch, type_, lens, new, G, D):
    c = Case(torch, type_, lens, 1, D, 16, seed=D)
    for name in "kv":
        s = c.scales[name].astype(np.float32)
        fine = np.isfinite(s)
        power = np.exp2(np.round(np.log2(np.abs(np.where(fine, s, 1.0)))))
        c.scales[name] = np.where(fine, np.sign(np.where(fine, s, 1.0)) * power, np.nan).astype(np.float16)
    c.upload()
    q_starts = np.arange(len(lens) + 1) * new
    q = np.random.default_rng(2).standard_normal((len(lens) * new, G, D)).astype(np.float32)
    scale = 1 / math.sqrt(D)
    got, lse, q = run_attend(c, q, q_starts, lens, "f16", None, scale)
    for s, n in enumerate(lens):
        seen = np.arange(n)[None, :] <= (n - new + np.arange(new))[:, None]
        k, v = c.dense("k", s)[:, 0], c.dense("v", s)[:, 0]
        rows = slice(q_starts[s], q_starts[s + 1])
        for hq in range(G):
            out, mag, ls, big = plain.attend(q[rows, hq].astype(np.float64), k, v, seen, scale)
            rel = 2.0 ** -20 * (1 + big[:, None])
            tol = 2 * rel * mag + 2.0 ** -11 * (np.abs(out) + 2 * rel * mag) + 2.0 ** -25
            err = np.abs(got[rows, hq] - out)
            assert (err <= tol).all(), (s, hq, float((err / tol).max()))
