"""Sampling on the GPU against the formula in 64 bits: the same token wherever u and top_p keep clear of the borders."""
import numpy as np
import pytest

from tests import plain_step as step
from tests.gpu_util import torch_mod

pytestmark = pytest.mark.gpu
CLEAR = 1e-8        # V * 2^-43 at V = 2^16: nearer to a border than this, the token may differ


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


def run(torch, dtype, z, t=None, k=None, p=None, q=None, u=None, pad=0, offset=0, logp=True, stream=None):
    """z: [R, V] on the GPU, of its type."""
    import block_quantized_matmul_gb300 as qmm

    R, V = z.shape
    buf = torch.full((offset + R * (V + pad),), 1000.0, dtype=z.dtype, device="cuda")
    rows = buf[offset:].view(R, V + pad)
    rows[:, :V] = z
    d = lambda a, ty: None if a is None else torch.from_numpy(np.array(a, dtype=ty)).cuda()  # noqa: E731
    tok = torch.full((R + 1,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((R + 1,), -7.0, device="cuda") if logp else None
    qmm.qmm_sample(dtype, rows, V + pad, R, V, d(t, np.float32), d(k, np.int32), d(p, np.float32), d(q, np.float32), d(u, np.float32), tok, lp, stream=stream)
    torch.cuda.synchronize()
    assert tok[-1] == -7 and (lp is None or lp[-1] == -7)
    return tok[:-1].cpu().numpy(), None if lp is None else lp[:-1].cpu().numpy()


def check(torch, dtype, z, t, k, p, q, u, **more):
    R = z.shape[0]
    full = lambda a, d: [d] * R if a is None else a  # noqa: E731
    tok, lp = run(torch, dtype, z, t, k, p, q, u, **more)
    z64 = z.double().cpu().numpy()
    f = np.float32
    close = 0
    for i in range(R):
        want, l, near = step.sample(z64[i], float(f(full(t, 1.0)[i])), int(full(k, 0)[i]), float(f(full(p, 1.0)[i])), float(f(full(q, 0.0)[i])), float(f(u[i])))
        if near < CLEAR:
            close += 1
            continue
        assert tok[i] == want, (i, tok[i], want, near)
        if lp is not None:
            assert abs(lp[i] - l) <= 2.0 ** -23 * abs(l) + 1e-8 or (np.isneginf(l) and np.isneginf(lp[i]))
    assert close <= R // 4


def logits(torch, dtype, R, V, seed, scale=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = scale * torch.randn(R, V, generator=gen, device="cuda")
    some = torch.randint(0, V, (R, 4), generator=gen, device="cuda")
    return z.scatter_add_(1, some, 4 + 3 * torch.rand(R, 4, generator=gen, device="cuda")).to(dtypes(torch)[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 2), (3, 7), (4, 100), (5, 1024), (3, 4097), (2, 16384), (2, 16400), (1, 32003), (40, 3000), (3, 65537)])
def test_sample(torch, dtype, R, V):
    rng = np.random.default_rng(V)
    z = logits(torch, dtype, R, V, V)
    for t, k, p, q in (([1.0] * R, None, None, None), (None, [min(V, 5)] * R, None, None), ([0.7] * R, None, [0.9] * R, None), ([1.3] * R, None, None, [0.02] * R),
                       (rng.uniform(0.3, 2, R), rng.integers(0, V + 3, R), rng.uniform(0.1, 1.05, R), rng.uniform(0, 0.2, R)),
                       ([0.0] * R, [3] * R, [0.5] * R, [0.5] * R)):
        check(torch, dtype, z, t, k, p, q, rng.random(R).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_cut_at_once_over_many_rows(torch, dtype):
    R, V = 64, 5000
    rng = np.random.default_rng(1)
    check(torch, dtype, logits(torch, dtype, R, V, 3, 1.5), rng.choice([0.0, 0.5, 1.0, 2.0, 10.0], R), rng.choice([0, -3, 1, 2, 50, 1000, 4999, 5000, 9999], R),
          rng.choice([1.0, 0.99, 0.5, 0.01, 0.0, -1.0, 2.0], R), rng.choice([0.0, 0.001, 0.3, 0.999, 1.0, 1.5, -1.0], R), rng.random(R))


@pytest.mark.parametrize("V", [123000, 128256, 129500])
def test_rows_in_few_large_slices(torch, V):
    """So many rows of 16-bit logits that each is taken in as few and large slices as fit, where they fit."""
    rng = np.random.default_rng(V)
    R = 80
    check(torch, "bf16", logits(torch, "bf16", R, V, 19), rng.choice([0.0, 0.7, 1.0, 1.3], R, p=[0.1, 0.3, 0.3, 0.3]), rng.choice([0, 1, 40, 3000], R), rng.choice([1.0, 0.95, 0.5], R),
          rng.choice([0.0, 0.01], R), rng.random(R).astype(np.float32))


@pytest.mark.parametrize("V", [4000, 130000])
def test_wide_cuts_and_flat_logits(torch, V):
    """Cuts that keep many tokens, where borders lie in the bulk."""
    R = 6
    rng = np.random.default_rng(2)
    z = logits(torch, "f32", R, V, 5, 0.3)
    check(torch, "f32", z, [1.0, 1.3, 0.8, 1.0, 5.0, 1.0], [0, V // 2, V - 1, 0, V // 3, 0], [0.95, 0.9, 0.5, 0.999, 0.99, 1.0], [0, 0, 0, 0.3, 0.2, 0.5], rng.random(R))


@pytest.mark.parametrize("top_p", [0.3, 0.9, 0.999])
def test_a_border_among_logits_that_are_all_low(torch, top_p):
    """One logit on top, and V - 1 around the level at which all together weigh as much as top_p leaves of it."""
    V, t = 30000, 0.7
    rng = np.random.default_rng(18)
    level = t * np.log(V / (1 - top_p))
    shifts = np.array([-3, -1, -0.3, -0.1, -0.03, -0.01, 0, 0.01, 0.03, 0.1, 0.3, 1, 3])
    z = 5 - level + t * shifts[:, None] + 0.02 * rng.standard_normal((len(shifts), V))
    z[:, 777] = 5
    z[:, 20000:20005] = 4.9 - np.arange(5)
    R = len(shifts)
    check(torch, "f32", torch.from_numpy(z.astype(np.float32)).cuda(), [t] * R, None, [top_p] * R, None, rng.random(R).astype(np.float32))
    check(torch, "f32", torch.from_numpy(z.astype(np.float32)).cuda(), [t] * R, [25000] * R, [top_p] * R, None, rng.random(R).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_ties_go_to_the_lowest_index(torch, dtype):
    """Few values: every cut falls among equal logits.  The shares are multiples of 1/64 of each other's, so sums are exact, and
    borders can be met: u and top_p are taken between them."""
    R, V = 12, 9000
    rng = np.random.default_rng(3)
    z = torch.from_numpy(rng.integers(0, 3, (R, V)).astype(np.float32)).to(dtypes(torch)[dtype]).cuda()
    z[3] = 1.0
    z[4] = -0.0
    z[4, ::2] = 0.0
    k = [0, 1, 5, 777, 4444, 8999, 3000, 6001, 2, 0, 0, 100]
    p = [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.4321, 0.9, 0.7, 0.12345, 0.98765, 0.5003]
    check(torch, dtype, z, [1.0] * R, k, p, None, (rng.integers(0, 1000, R) + 0.437) / 1000)
    tok, _ = run(torch, dtype, z, [0.0] * R, u=[0.9] * R)
    np.testing.assert_array_equal(tok, z.float().argmax(1).cpu().numpy() if dtype == "f32" else [int(np.argmax(r)) for r in z.float().cpu().numpy()])


def test_masked_logits(torch):
    """-inf, the lowest finite value, NaN and +inf among the logits; rows of nothing else."""
    V = 3000
    lowest = torch.finfo(torch.float32).min
    z = logits(torch, "f32", 10, V, 7)
    z[0, 5:] = -np.inf
    z[1, :] = -np.inf
    z[2, :] = np.nan
    z[3, :] = lowest                       # all alike: any token, equally likely
    z[4, 10:] = lowest
    z[5, 3] = z[5, 77] = np.inf            # one of the two
    z[6, ::2] = np.nan
    z[7, 1:] = -np.inf
    z[8, :] = -np.inf
    z[8, V - 1] = lowest
    z[9, 2] = np.inf
    z[9, 1] = lowest
    u = np.linspace(0.03, 0.97, 10).astype(np.float32)
    for k, p, q in ((None, None, None), ([4] * 10, None, None), (None, [0.6] * 10, None), ([50] * 10, [0.9] * 10, [0.01] * 10)):
        check(torch, "f32", z, [0.9] * 10, k, p, q, u)
    tok, lp = run(torch, "f32", z, [0.9] * 10, u=u)
    assert tok[1] == -1 and tok[2] == -1 and np.isneginf(lp[1]) and np.isneginf(lp[2]) and tok[7] == 0 and tok[8] == V - 1
    assert abs(lp[3] + np.log(V)) < 1e-5 and abs(lp[5] + np.log(2)) < 1e-6 and tok[5] in (3, 77)
    tok, lp = run(torch, "f32", z, [0.0] * 10, u=u)
    assert tok[1] == -1 and np.isneginf(lp[1]) and tok[5] == 3 and tok[8] == V - 1 and tok[9] == 2 and lp[5] == 0


def test_random_numbers_at_the_ends(torch):
    """u = 0 takes the first kept token, u next to 1 the last, and what lies outside counts as the nearest of those."""
    V = 700
    z = logits(torch, "f32", 1, V, 9).repeat(7, 1)
    u = np.array([0.0, -1.0, np.nan, 1.0, 2.0, np.nextafter(np.float32(1), np.float32(0)), 1e-42], np.float32)
    tok, _ = run(torch, "f32", z, [1.0] * 7, k=[50] * 7, u=u)
    kept = np.sort(np.argsort(-z[0].cpu().numpy(), kind="stable")[:50])
    assert tok[0] == tok[1] == tok[2] == tok[6] == kept[0] and tok[3] == tok[4] == tok[5] == kept[-1]


def test_extreme_temperatures(torch):
    V = 2000
    z = logits(torch, "f32", 8, V, 11)
    t = [1e-42, 1e-30, 1e-4, 1e4, 1e30, np.inf, np.nan, -1.0]
    check(torch, "f32", z, t, None, None, None, np.linspace(0.1, 0.9, 8))
    check(torch, "f32", z, t, [100] * 8, [0.77] * 8, None, np.linspace(0.1, 0.9, 8))
    wide = z * 1e37
    check(torch, "f32", wide, t, None, [0.9] * 8, None, np.linspace(0.1, 0.9, 8))


@pytest.mark.parametrize("pad,offset", [(0, 0), (4, 0), (1, 0), (3, 1), (8, 4)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_strides_and_alignment(torch, dtype, pad, offset):
    rng = np.random.default_rng(13)
    check(torch, dtype, logits(torch, dtype, 5, 8195, 13), [1.0] * 5, [0, 9, 0, 300, 0], [1, 1, 0.8, 0.9, 1], None, rng.random(5), pad=pad, offset=offset, logp=False)


@pytest.mark.parametrize("dtype,V", [("f32", 500000), ("f32", 1 << 20), ("bf16", 1 << 20)])
def test_vocabularies_beyond_shared_memory(torch, dtype, V):
    rng = np.random.default_rng(17)
    check(torch, dtype, logits(torch, dtype, 4, V, 17), [1.0, 0.6, 1.0, 1.0], [0, 0, 40, 70000], [1.0, 0.9, 0.95, 0.99], [0, 0, 0, 1e-4], rng.random(4))


def test_shares(torch):
    """Over evenly spread random numbers every token comes as often as its share says (the counts of an inverse
    distribution differ from n * share by less than one)."""
    V, n = 300, 4096
    z = logits(torch, "f32", 1, V, 19)
    u = (np.arange(n) + 0.5) / n
    tok, lp = run(torch, "f32", z.repeat(n, 1), [1.5] * n, k=[60] * n, u=u)
    w = np.exp((z[0].double().cpu().numpy() - float(z.max())) / 1.5)
    keep = np.argsort(-z[0].cpu().numpy(), kind="stable")[:60]
    share = np.zeros(V)
    share[keep] = w[keep] / w[keep].sum()
    assert (np.abs(np.bincount(tok, minlength=V) - n * share) <= 1 + 1e-6).all()
    assert np.abs(lp - np.log(share[tok])).max() <= 1e-6


def test_the_same_again_on_other_streams_and_in_graphs(torch):
    import block_quantized_matmul_gb300 as qmm

    R, V = 20, 40000
    rng = np.random.default_rng(23)
    z = logits(torch, "f32", R, V, 23)
    u = rng.random(R).astype(np.float32)
    args = dict(t=[1.0] * R, k=[0] * 10 + [100] * 10, p=[0.95] * R, u=u)
    want, lp = run(torch, "f32", z, **args)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        got, l2 = run(torch, "f32", z, stream=s, **args)
        np.testing.assert_array_equal(got, want)
        np.testing.assert_array_equal(l2, lp)
    d = lambda a, ty: torch.from_numpy(np.array(a, dtype=ty)).cuda()  # noqa: E731
    t, k, p, ud = d([1.0] * R, np.float32), d(args["k"], np.int32), d(args["p"], np.float32), d(u, np.float32)
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_sample("f32", z, V, R, V, t, k, p, None, ud, tok, None)
    u2 = rng.random(R).astype(np.float32)
    for numbers, w in ((u, want), (u2, run(torch, "f32", z, **(args | {"u": u2}))[0])):
        ud.copy_(torch.from_numpy(numbers))
        graph.replay()
        np.testing.assert_array_equal(tok.cpu().numpy(), w)
