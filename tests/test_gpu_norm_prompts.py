"""The norms over so many rows that the kernels of prompts take them (more than one an SM), in each class of widths, with the types that
the compiler knows and those that it does not."""
import numpy as np
import pytest

from tests.test_gpu_norm import rows, run, torch  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
R = 160

# the widest row of each class, the first of the next, and rows that the vectorised path does not take
WIDTHS = [8, 256, 264, 500, 512, 520, 1024, 1032, 2047, 2048, 2056, 3001, 4096, 4104, 8191, 8192, 8200, 14336, 16384, 16392, 32768]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f16", "f16", "f16"), ("f32", "f32", "f32"), ("f16", "f32", "bf16")]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("xdt,hdt,ydt", TYPES)
def test_widths(torch, N, xdt, hdt, ydt):  # noqa: F811
    run(torch, np.random.default_rng(N), R, N, xdt, hdt, ydt, gate="all")


@pytest.mark.parametrize("N", [512, 1024, 2048, 4096, 8192])
@pytest.mark.parametrize("hdt", ["bf16", "f32"])
def test_parts_left_out(torch, N, hdt):  # noqa: F811
    rng = np.random.default_rng(N + 1)
    run(torch, rng, R, N, "bf16", hdt, "bf16", post=False, gate="none")
    run(torch, rng, R, N, "bf16", hdt, "bf16", gate="rows", pre=False)
    run(torch, rng, R, N, "bf16", hdt, "bf16", with_x=False)
    run(torch, rng, R, N, "bf16", hdt, "bf16", in_place=True)
    run(torch, rng, R, N, "bf16", hdt, "bf16", pad=16)
    run(torch, rng, R, N, "bf16", hdt, "bf16", pad=3, offset=1)


@pytest.mark.parametrize("N", [32, 256, 512, 1024, 1056, 2048, 4096, 4128, 8192, 16384, 32768])
@pytest.mark.parametrize("form", ["q8", "mx4"])
@pytest.mark.parametrize("xdt,hdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("pad", [0, 1])
def test_operands(torch, N, form, xdt, hdt, pad):  # noqa: F811
    """Those of the library's quantizers on the same rows, bit for bit."""
    import block_quantized_matmul_gb300 as qmm

    rng = np.random.default_rng(N)
    x, h = rows(torch, rng, R, N, xdt, pad), rows(torch, rng, R, N, hdt, pad)
    h[3, :32] = 0
    x[3, :32] = 0
    w = torch.rand(N, device="cuda") + 0.5
    args = (xdt, x, N + pad, hdt, h, N + pad, R, N, w, x, N + pad, 0.5, w, 1e-6)
    ho, ho2, y = torch.empty(R, N, dtype=h.dtype, device="cuda"), torch.empty(R, N, dtype=h.dtype, device="cuda"), torch.empty(R, N, device="cuda")
    if form == "q8":
        got = [torch.full((R, N), 99, dtype=torch.int8, device="cuda"), torch.full((R, N // 32), -1, dtype=torch.int16, device="cuda")]
        want = [torch.empty_like(t) for t in got]
        qmm.qmm_norm_q8(*args, ho2, N, *got)
    else:
        got = [torch.full((R, N // 2), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((qmm.mx4_scales_size(R, N),), 0xA5, dtype=torch.uint8, device="cuda")]
        want = [torch.full_like(t, 0xA5) for t in got]
        qmm.qmm_norm_mx4(*args, ho2, N, *got)
    qmm.qmm_norm(*args, ho, N, "f32", y, N)
    if form == "q8":
        qmm.qmm_quantize_act(y, R, N, N, *want)
    else:
        qmm.qmm_mx4_quantize("f32", y, R, N, N, *want)
    assert torch.equal(ho, ho2)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_many_rows_are_the_few(torch):  # noqa: F811
    """A row's results do not depend on how many are taken with it, but for the order of its sums: within a rounding of y's type of
    each other, whichever kernel takes them."""
    import block_quantized_matmul_gb300 as qmm

    for N in (1024, 2048, 4096, 8192):
        rng = np.random.default_rng(N)
        x, h = rows(torch, rng, 400, N, "bf16", 0), rows(torch, rng, 400, N, "f32", 0)
        w = torch.rand(N, device="cuda") + 0.5
        out = []
        for part in (400, 100):
            y, ho = torch.empty(400, N, dtype=torch.bfloat16, device="cuda"), torch.empty(400, N, device="cuda")
            for a in range(0, 400, part):
                qmm.qmm_norm("bf16", x[a:], N, "f32", h[a:], N, part, N, w, None, 0, 1.0, w, 1e-6, ho[a:], N, "bf16", y[a:], N)
            out.append((y.double(), ho.double()))
        (y0, h0), (y1, h1) = out
        e = 2.0 ** -24 * (N / 16 + 24)
        # h' = h + x r w: twice the error of r, and a rounding each
        assert ((h0 - h1).abs() <= 2 * (e + 2.0 ** -24) * ((h0 - h.double()).abs() + h.double().abs())).all()
        # y's two results lie at most two half steps of bf16 and the errors before them apart
        assert ((y0 - y1).abs() <= (2 * 2.0 ** -8 + 8 * e) * y0.abs() + 8 * e).all()
