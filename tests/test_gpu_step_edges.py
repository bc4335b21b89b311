"""The calls of a decode step where offsets pass 32 bits, where calls run at the same time, and over very many rows."""
import numpy as np
import pytest

from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, device
from tests.test_gpu_norm import run as run_norm
from tests.test_gpu_sample import logits, run as run_sample
from tests.test_gpu_sparse import gpu_attend, gpu_bounds, gpu_select

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
def test_pages_far_into_a_pool(torch, type_):
    """The same pages under numbers whose offsets in the caches, then in the bounds, pass 2^32 bytes give the same results."""
    import block_quantized_matmul_gb300 as qmm

    lens, news, H, D, P = [9000, 700], [1, 2], 8, 128, 256
    c = Case(torch, type_, lens, H, D, P, seed=31).upload()
    q = np.random.default_rng(32).standard_normal((3, 4 * H, D)).astype(np.float32)
    bounds = gpu_bounds(c, lens)
    chosen, _ = gpu_select(c, bounds, q, news, "bf16", None, 1, 2, 6)
    want, lse, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen)

    small, table, pages = c.n_pages, c.table.copy(), c.pages
    page = qmm.cache_page_size(type_, H, D, P)
    many = 2 ** 32 // page + small + 1
    far = np.random.default_rng(33).permutation(small) + (many - small)
    at = device(torch, far.astype(np.int64))
    near = {}
    for name in ("k_cache", "v_cache"):
        near[name] = getattr(c, name)
        big = torch.empty(many, page, dtype=torch.uint8, device="cuda")
        big[at] = near[name].view(torch.uint8).reshape(small, page)
        setattr(c, name, big)
    c.n_pages, c.pages = many, device(torch, np.where(table >= 0, far[np.clip(table, 0, small - 1)], table).astype(np.int32))
    again = gpu_bounds(c, lens)
    used = np.unique(np.concatenate([table[s, : (n + P - 1) // P] for s, n in enumerate(lens)]))
    assert torch.equal(again[device(torch, far[used].astype(np.int64))], bounds[device(torch, used.astype(np.int64))])
    got, lse2, _ = gpu_attend(c, q, news, "bf16", None, 0.1, chosen)
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(lse2, lse)
    del again, big
    for name, b in near.items():
        setattr(c, name, b)
    torch.cuda.empty_cache()

    many = 2 ** 32 // qmm.cache_bounds_size(H, D) + small + 1
    far += many - small - far.min()
    at = device(torch, far.astype(np.int64))
    big = torch.empty((many,) + tuple(bounds.shape[1:]), dtype=torch.uint8, device="cuda")
    big[at] = bounds
    c.n_pages, c.pages = many, device(torch, np.where(table >= 0, far[np.clip(table, 0, small - 1)], table).astype(np.int32))
    assert torch.equal(gpu_select(c, big, q, news, "bf16", None, 1, 2, 6)[0], chosen)


def test_calls_at_the_same_time(torch):
    """Choice and attention, norms and samples under way on three streams, each with its own workspaces."""
    import block_quantized_matmul_gb300 as qmm

    H, Hq, D, P, budget = 2, 8, 128, 16, 9
    work = []
    for i in range(3):
        lens = [3000 + 500 * i, 100 * i + 40, 1]
        c = Case(torch, "q8_0", lens, H, D, P, seed=40 + i).upload()
        bounds = gpu_bounds(c, lens)
        gen = torch.Generator(device="cuda").manual_seed(50 + i)
        q = torch.randn(3, Hq * D, generator=gen, device="cuda").bfloat16()
        starts, kv = device(torch, np.arange(4, dtype=np.int32)), device(torch, np.array(lens, np.int32))
        need = qmm.cache_select_workspace_size(3, H, P, P * c.table.shape[1]), qmm.cache_attend_chosen_workspace_size(3, H, Hq, D, P, budget)
        ws = [torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda") for n in need]
        z = logits(torch, "f32", 5 + 40 * i, 30000 + 7 * i, 60 + i)
        R, V = z.shape
        u, p = torch.rand(R, generator=gen, device="cuda"), torch.full((R,), 0.9, device="cuda")
        out = dict(chosen=torch.zeros(3, H, budget, dtype=torch.int32, device="cuda"), out=torch.zeros_like(q), lse=torch.zeros(3, Hq, device="cuda"),
                   h=torch.zeros_like(q), y=torch.zeros_like(q), tokens=torch.zeros(R, dtype=torch.int32, device="cuda"), logp=torch.zeros(R, device="cuda"))

        def step(stream, c=c, bounds=bounds, q=q, starts=starts, kv=kv, need=need, ws=ws, z=z, u=u, p=p, R=R, V=V, out=out):
            ld = c.table.shape[1]
            qmm.qmm_cache_select(bounds, c.n_pages, P, H, D, c.pages, ld, starts, kv, 3, "bf16", q, Hq * D, 3, Hq, None, 1, P * ld, 1, 2, budget,
                                 out["chosen"], ws[0], ws[0].numel(), stream=stream)
            qmm.qmm_cache_attend_chosen("q8_0", c.k_cache, c.v_cache, c.n_pages, P, H, D, c.pages, ld, starts, kv, 3, "bf16", q, Hq * D, 3, Hq, None, 0.1,
                                        out["chosen"], budget, out["out"], Hq * D, out["lse"], ws[1], need[1], stream=stream)
            qmm.qmm_norm("bf16", out["out"], Hq * D, "bf16", q, Hq * D, 3, Hq * D, None, None, 0, 1.0, None, 1e-6, out["h"], Hq * D, "bf16", out["y"], Hq * D,
                         stream=stream)
            qmm.qmm_sample("f32", z, V, R, V, None, None, p, None, u, out["tokens"], out["logp"], stream=stream)

        work.append((step, out))
    alone = []
    for step, out in work:
        step(None)
        torch.cuda.synchronize()
        alone.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        for _, out in work:
            for v in out.values():
                v.zero_()
        torch.cuda.synchronize()
        for _ in range(8):
            for (step, _), s in zip(work, streams):
                step(s)
        torch.cuda.synchronize()
        for (_, out), want in zip(work, alone):
            for k, v in out.items():
                assert torch.equal(v, want[k]), k


def test_very_many_rows(torch):
    run_norm(torch, np.random.default_rng(70), 70000, 8, xdt="f32", hdt="f32", ydt="f32")
    z = logits(torch, "bf16", 70000, 40, 71, 1.0)
    z64 = z.double().cpu().numpy()
    np.testing.assert_array_equal(run_sample(torch, "bf16", z, t=[0.0] * 70000, u=[0.5] * 70000)[0], z64.argmax(-1))
    tok, lp = run_sample(torch, "bf16", z, u=[0.0] * 70000)                        # the first of all (none is 2^-43 of the largest)
    assert (tok == 0).all()
    top = z64.max(-1)
    want = z64[:, 0] - top - np.log(np.exp(z64 - top[:, None]).sum(-1))
    assert (np.abs(lp - want) <= 2.0 ** -23 * np.abs(want) + 1e-8).all()
