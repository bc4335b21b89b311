"""Cuts of the sampling where the weights of neighbouring logits are so close that they cannot be told apart."""
import numpy as np
import pytest

from tests.test_gpu_sample import run, torch  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
f32 = np.float32


def test_the_first_token_that_min_p_takes_ends_the_line(torch):  # noqa: F811
    """The weights of z[20] and z[30] are 5.942521966e-5 of the largest, 1e-15 apart, which is less than their steps of 2^-43, and min_p
    lies as near: to take neither, one or both is within the stated error.  Whatever is kept is a run from
    the first in rank on: index 7 alone, with 20, or with 20 and 30, never with 30 alone and never twice."""
    z = np.full((5, 100), -5, f32)
    z[:, 7], z[:, 20], z[:, 30] = 7.78449821472168, -0.0001353803090751171, -0.00013538032362703234
    u = np.array([0.0, 0.25, 0.499, 0.501, 0.99], f32)
    w = np.exp((z[0].astype(np.float64) - z[0, 7]) / float(f32(0.8)))
    tok, lp = run(torch, "f32", torch.from_numpy(z).cuda(), [0.8] * 5, [10] * 5, None, [5.942521966062486e-05] * 5, u)
    assert (tok == 7).all()                                     # all others together are less than 1 - 0.99 of it
    # ln of 1 / (1 + j w) for j = 0, 1, 2, rounded once but for 2^-30 of itself
    j = np.rint((np.exp(-lp.astype(np.float64)) - 1) / w[20])
    assert (j == j[0]).all() and j[0] in (0, 1, 2)
    np.testing.assert_allclose(lp, -np.log1p(j * w[20]), rtol=2.0 ** -23, atol=1e-8)


@pytest.mark.parametrize("top,t", [(7.7845, 0.8), (3.0, 1.0), (0.5, 1.3), (11.0, 1.0)])
@pytest.mark.parametrize("top_p", [1.0, 0.9999999])
def test_a_border_among_weights_that_lie_within_their_error(torch, top, t, top_p):  # noqa: F811
    """Twenty logits around 0 whose weights differ by less than the error of a weight, and min_p around them: for one row of
    parameters all random numbers see the same kept tokens, the first in rank of the twenty."""
    V, n, few = 200, 20, 48
    rng = np.random.default_rng(int(10 * top))
    z = np.full(V, -9, f32)
    z[11] = top
    at = np.sort(rng.choice(np.arange(20, V), n, replace=False))
    z[at] = (1e-12 * rng.standard_normal(n)).astype(f32)
    w = float(np.exp(-float(f32(top)) / float(f32(t))))
    rank = at[np.argsort(-z[at], kind="stable")]
    u = ((np.arange(few) + 0.5) / few).astype(f32)
    # fp32 numbers around w, near together: every border within 2^-24 of it
    q = [f32(w)]
    for _ in range(3):
        q = [np.nextafter(q[0], f32(0))] + q + [np.nextafter(q[-1], f32(1))]
    rows = len(q) * few
    tok, lp = run(torch, "f32", torch.from_numpy(np.tile(z, (rows, 1))).cuda(), [t] * rows, [n + 1] * rows, [top_p] * rows, np.repeat(q, few), np.tile(u, len(q)))
    tok, lp = tok.reshape(-1, few), lp.reshape(-1, few).astype(np.float64)
    for i in range(len(q)):
        # how many of the twenty are kept, from the share of any token: 1 / total or w / total
        share = np.exp(-lp[i]) * np.where(tok[i] == 11, 1.0, w)
        j = np.rint((share - 1) / w)
        assert (j == j[0]).all() and 0 <= j[0] <= n
        kept = np.sort(np.append(rank[: int(j[0])], 11))
        upto = np.cumsum(np.where(kept == 11, 1.0, w))
        for k in range(few):
            edge = np.abs(upto / upto[-1] - float(u[k])).min()
            if edge > 1e-8:
                assert tok[i, k] == kept[int((upto <= float(u[k]) * upto[-1]).sum())], (i, k, j[0])


@pytest.mark.parametrize("seed", range(4))
def test_weights_keep_their_stated_distance(torch, seed):  # noqa: F811
    """Two logits: a min_p of the lower one's weight, less (more) than 9/8 of 2^-43 and 2^-34 of itself, keeps (drops) it.  With u = 0 the
    token is the lower one, the first index, exactly when it is kept.  min_p in fp32 is rounded away from the weight."""
    n = 20000
    rng = np.random.default_rng(seed)
    t = np.exp(rng.uniform(-1.5, 1.5, n)).astype(f32)
    top = rng.uniform(-20, 20, n).astype(f32)
    # all powers of two down to 2^-43, 2^-14 to 2^-18 the most
    y = np.where(rng.random(n) < 0.5, rng.uniform(0, 43, n), rng.uniform(13, 18, n))
    z = (top - y * np.log(2) * t.astype(np.float64)).astype(f32)
    w = np.exp((z.astype(np.float64) - top) / t) * 2.0 ** 43
    err = 9 / 8 + 2.0 ** -34 * w * (1 + 1e-3)                   # (fp64's own exponential: 2^-50)
    low, high = np.floor(w - err) * 2.0 ** -43, (w + err) * 2.0 ** -43
    q0, q1 = low.astype(f32), high.astype(f32)
    q0 = np.where(q0 > low, np.nextafter(q0, f32(0)), q0)
    q1 = np.where(q1 <= high, np.nextafter(q1, f32(2)), q1)
    use = (low > 0) & (q1 < 1) & (z < top)
    assert use.sum() > n // 2
    rows = torch.from_numpy(np.stack([z, top], 1)[use]).cuda()
    m = len(rows)
    for q, want in ((q0, 0), (q1, 1)):
        tok, _ = run(torch, "f32", rows, t[use], None, None, q[use], np.zeros(m, f32))
        assert (tok == want).all(), (want, np.flatnonzero(tok != want)[:5])
