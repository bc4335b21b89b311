"""The norms around a block on the GPU, against the formula in 64 bits; the quantized forms against the library's own
quantizers, bit for bit."""
import numpy as np
import pytest

from tests import plain_step as step
from tests.gpu_util import torch_mod

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # one rounding, relative (half a step)
TINY = {"f32": 1e-40, "f16": 2.0 ** -25, "bf16": 1e-40}                # half a step of subnormal numbers


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


def rows(torch, rng, r, n, dtype, pad, scale=1.0, offset=0):
    """A [r, n] view of a wider buffer that starts `offset` elements in."""
    ld = n + pad
    buf = torch.full((offset + r * ld,), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    v = buf[offset:].view(r, ld)[:, :n]
    v.copy_(torch.from_numpy((scale * rng.standard_normal((r, n))).astype(np.float32)).cuda())
    return v


def tolerance(n, x, h, w_post, gate, scale, w_pre, h_want, y_want, hdt, ydt):
    """fp32 steps: a mean of n squares (pairwise over at least 8 lanes, at most n/8 + 12 roundings of 2^-24, halved by the root), a
    division, a root, products and a sum: each 2^-24 of the largest number involved.  h' takes one rounding of its type; y takes the
    change of h' over a rounding border (one full step of its type) into account."""
    e = 2.0 ** -24 * (n / 16 + 24)
    part = np.abs(h_want) if x is None else np.abs(h) + np.abs(h_want - h)
    tol_h = e * part + HALF[hdt] * np.abs(h_want) + TINY[hdt]
    rms = np.sqrt((h_want ** 2).mean(-1, keepdims=True) + 1e-30)
    moved = e * part + 2 * HALF[hdt] * np.abs(h_want) + TINY[hdt]           # of the h' that y is computed from
    w = 1.0 if w_pre is None else np.abs(w_pre)
    # the row's own mean moves by at most the largest relative move of its elements
    tol_y = moved / rms * w + (e + 2 * HALF[hdt] + (moved.max(-1, keepdims=True) / rms)) * np.abs(y_want) + HALF[ydt] * np.abs(y_want) + TINY[ydt]
    return tol_h, tol_y


def run(torch, rng, R, N, xdt="bf16", hdt="f32", ydt="bf16", post=True, gate="rows", pre=True, with_x=True, pad=0, offset=0, eps=1e-6, in_place=False):
    import block_quantized_matmul_gb300 as qmm

    x = rows(torch, rng, R, N, xdt, pad, 0.5, offset) if with_x else None
    h = rows(torch, rng, R, N, hdt, pad, 2.0, offset)
    g = None if gate == "none" or not with_x else rows(torch, rng, R if gate == "rows" else 1, N, xdt, pad, 1.0, offset)
    wp = torch.from_numpy((1 + 0.1 * rng.standard_normal(N)).astype(np.float32)).cuda() if post and with_x else None
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(N)).astype(np.float32)).cuda() if pre else None
    h64 = h.double().cpu().numpy()
    ho = h if in_place else torch.full((R, N + pad), -7.0, dtype=h.dtype, device="cuda")[:, :N]
    y = torch.full((R, N + pad), -7.0, dtype=dtypes(torch)[ydt], device="cuda")[:, :N]
    qmm.qmm_norm(xdt, x, N + pad, hdt, h, N + pad, R, N, wp, g, N + pad if gate == "rows" else 0, 0.75, w, eps, ho, N + pad, ydt, y, N + pad)
    torch.cuda.synchronize()
    if pad and not in_place:
        assert (ho._base[:, N:] == -7).all() and (y._base[:, N:] == -7).all()
    n64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    rounded = lambda v: torch.from_numpy(v).to(dtypes(torch)[hdt]).double().numpy()  # noqa: E731
    exact, _ = step.norm(n64(x), h64, n64(wp), n64(g), 0.75, n64(w), eps, lambda v: v)
    h_want, _ = step.norm(n64(x), h64, n64(wp), n64(g), 0.75, n64(w), eps, rounded)
    # y from the h' that was stored
    _, y_want = step.norm(None, n64(ho), None, None, 1.0, n64(w), eps, lambda v: v)
    tol_h, _ = tolerance(N, n64(x), h64, n64(wp), n64(g), 0.75, n64(w), h_want, y_want, hdt, ydt)
    assert (np.abs(n64(ho) - exact) <= tol_h).all(), np.abs(n64(ho) - exact).max()
    e = 2.0 ** -24 * (N / 16 + 24)
    assert (np.abs(n64(y) - y_want) <= (e + HALF[ydt]) * np.abs(y_want) + TINY[ydt]).all()
    return x, h, ho, y


@pytest.mark.parametrize("R,N", [(1, 1), (3, 5), (2, 31), (5, 32), (9, 128), (4, 250), (7, 256), (3, 500), (2, 1000), (1, 1024), (3, 1025), (2, 2048), (1, 4096),
                                 (5, 4099), (2, 8192), (1, 14336), (2, 16384), (1, 20000), (1, 32768)])
@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "rows"), (True, "all")])
def test_norm_sizes(torch, R, N, post, gate):
    run(torch, np.random.default_rng(N), R, N, post=post, gate=gate)


@pytest.mark.parametrize("xdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ydt", ["f32", "f16", "bf16"])
def test_norm_types(torch, xdt, hdt, ydt):
    run(torch, np.random.default_rng(1), 3, 768, xdt, hdt, ydt)
    run(torch, np.random.default_rng(2), 2, 2056, xdt, hdt, ydt, gate="all", post=False)


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (8, 0), (3, 5), (16, 16)])
def test_norm_strides_and_alignment(torch, pad, offset):
    run(torch, np.random.default_rng(3), 4, 640, pad=pad, offset=offset)
    run(torch, np.random.default_rng(4), 2, 3000, hdt="bf16", pad=pad, offset=offset)


def test_norm_without_parts(torch):
    rng = np.random.default_rng(5)
    run(torch, rng, 6, 320, pre=False, gate="none")
    x, h, ho, y = run(torch, rng, 6, 4096, with_x=False)
    assert torch.equal(h, ho)
    run(torch, rng, 6, 4096, in_place=True, hdt="bf16")


def test_norm_alone_writes_no_stream(torch):
    import block_quantized_matmul_gb300 as qmm

    h = torch.randn(3, 96, device="cuda")
    y = torch.empty(3, 96, device="cuda")
    qmm.qmm_norm("bf16", None, 0, "f32", h, 96, 3, 96, None, None, 0, 1.0, None, 0.0, None, 0, "f32", y, 96)
    want = h.double() / h.double().pow(2).mean(1, keepdim=True).sqrt()
    assert (y.double() - want).abs().max() <= 2.0 ** -24 * 40 * want.abs().max()


def test_norm_rows_of_zeros(torch):
    import block_quantized_matmul_gb300 as qmm

    z = torch.zeros(2, 2048, dtype=torch.bfloat16, device="cuda")
    ho, y = torch.full_like(z, 7), torch.full_like(z, 7)
    qmm.qmm_norm("bf16", z, 2048, "bf16", z, 2048, 2, 2048, torch.ones(2048, device="cuda"), None, 0, 1.0, None, 1e-6, ho, 2048, "bf16", y, 2048)
    assert (ho == 0).all() and (y == 0).all()


def test_an_infinity_stays_in_its_row(torch):
    import block_quantized_matmul_gb300 as qmm

    h = torch.randn(3, 512, device="cuda")
    h[1, 7] = float("inf")
    y = torch.empty_like(h)
    qmm.qmm_norm("f32", None, 0, "f32", h, 512, 3, 512, None, None, 0, 1.0, None, 1e-6, None, 0, "f32", y, 512)
    assert torch.isfinite(y[[0, 2]]).all() and torch.isnan(y[1, 7]) and (y[1, :7] == 0).all()


@pytest.mark.parametrize("R,N", [(1, 32), (3, 96), (2, 160), (5, 256), (2, 1024), (130, 544), (1, 4096), (3, 4128), (2, 14336), (1, 32768)])
@pytest.mark.parametrize("form", ["q8", "mx4"])
@pytest.mark.parametrize("pad", [0, 1])
def test_quantized_forms_are_the_quantizers_of_the_rows(torch, R, N, form, pad):
    import block_quantized_matmul_gb300 as qmm

    rng = np.random.default_rng(N + R)
    x, h = rows(torch, rng, R, N, "bf16", pad), rows(torch, rng, R, N, "f32", pad)
    h[0, :32] = 0
    x[0, :32] = 0
    w = torch.rand(N, device="cuda") + 0.5
    args = ("bf16", x, N + pad, "f32", h, N + pad, R, N, w, None, 0, 0.5, w, 1e-6)
    ho, y = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    ho2 = torch.empty_like(ho)
    qmm.qmm_norm(*args, ho, N, "f32", y, N)
    if form == "q8":
        got = [torch.full((R, N), 99, dtype=torch.int8, device="cuda"), torch.full((R, N // 32), -1, dtype=torch.int16, device="cuda")]
        want = [torch.empty_like(t) for t in got]
        qmm.qmm_norm_q8(*args, ho2, N, *got)
        qmm.qmm_quantize_act(y, R, N, N, *want)
    else:
        got = [torch.full((R, N // 2), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((qmm.mx4_scales_size(R, N),), 0xA5, dtype=torch.uint8, device="cuda")]
        want = [torch.full_like(t, 0xA5) for t in got]
        qmm.qmm_norm_mx4(*args, ho2, N, *got)
        qmm.qmm_mx4_quantize("f32", y, R, N, N, *want)
    assert torch.equal(ho, ho2)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_operands_go_into_the_products(torch):
    """norm -> Q8_0 operand -> qmm_matmul, and norm -> MX4 operand -> qmm_mx4_matmul, captured and replayed with other rows."""
    import block_quantized_matmul_gb300 as qmm

    R, N, M = 4, 512, 96
    gen = torch.Generator(device="cuda").manual_seed(0)
    wt = torch.randn(M, N, generator=gen, device="cuda") / 20
    tiled = torch.empty(qmm.tiled_size("q8_0", N, M), dtype=torch.uint8, device="cuda")
    flat = torch.empty(qmm.flat_size("q8_0", N, M), dtype=torch.uint8, device="cuda")
    qmm.qmm_quantize_weight("q8_0", wt, M, N, N, flat)
    qmm.qmm_repack("q8_0", flat, N, M, tiled)
    wc, ws = torch.empty(qmm.mx4_codes_size(M, N), dtype=torch.uint8, device="cuda"), torch.empty(qmm.mx4_scales_size(M, N), dtype=torch.uint8, device="cuda")
    qmm.qmm_mx4_quantize("f32", wt, M, N, N, wc, ws)
    x, h, w = (torch.randn(*s, generator=gen, device="cuda") for s in ((R, N), (R, N), (N,)))
    ho = torch.empty_like(h)
    a_q, a_d = torch.empty(R, N, dtype=torch.int8, device="cuda"), torch.empty(R, N // 32, dtype=torch.int16, device="cuda")
    c, sc = torch.empty(R, N // 2, dtype=torch.uint8, device="cuda"), torch.zeros(qmm.mx4_scales_size(R, N), dtype=torch.uint8, device="cuda")
    y1, y2 = torch.empty(R, M, device="cuda"), torch.empty(R, M, device="cuda")
    args = ("f32", x, N, "f32", h, N, R, N, w, None, 0, 1.0, w, 1e-6, ho, N)

    def chain():
        qmm.qmm_norm_q8(*args, a_q, a_d)
        qmm.qmm_matmul("q8_0", tiled, N, M, a_q, a_d, R, y1, M)
        qmm.qmm_norm_mx4(*args, c, sc)
        qmm.qmm_mx4_matmul(wc, ws, N, M, c, sc, R, "f32", y2, M)

    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    x.normal_(generator=gen)
    graph.replay()
    b = x.double() * torch.rsqrt(x.double().pow(2).mean(1, keepdim=True) + 1e-6) * w.double()
    s = h.double() + b
    y = s * torch.rsqrt(s.pow(2).mean(1, keepdim=True) + 1e-6) * w.double()
    want = y @ wt.double().t()
    for got, share in ((y1, 0.02), (y2, 0.3)):          # blocks of 8 bits on both sides; of 4 bits on both
        assert (got.double() - want).norm() <= share * want.norm()
