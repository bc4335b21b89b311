"""The quantized forms of the norm on rows that hold infinities and NaN, against the library's quantizers on the same rows, bit for
bit."""
import numpy as np
import pytest

from tests.test_gpu_norm import torch  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["q8", "mx4"])
@pytest.mark.parametrize("N,pad", [(32, 0), (96, 0), (512, 1), (4096, 0), (8192, 0)])
def test_rows_with_infinities_and_nan(torch, form, N, pad):  # noqa: F811
    """One of each in the stream (the whole row's norm follows from it), in the weights (one element of a block, and a whole block), and in x."""
    import block_quantized_matmul_gb300 as qmm

    R = 6
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, h = (torch.randn(R, N + pad, generator=gen, device="cuda") for _ in range(2))
    h[0, 7], h[1, N - 1], h[2, 5] = float("inf"), -float("inf"), float("nan")
    x[3, 3] = float("nan")
    w = torch.rand(N, generator=gen, device="cuda") + 0.5
    w[N - 2], w[9], w[11] = float("nan"), float("inf"), 0.0
    if N > 64:
        w[32:64] = float("nan")
    args = ("f32", x, N + pad, "f32", h, N + pad, R, N, None, None, 0, 0.5, w, 1e-6)
    ho, ho2, y = (torch.empty(R, N, device="cuda") for _ in range(3))
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
    assert torch.equal(ho.view(torch.int32), ho2.view(torch.int32)) and torch.isnan(y).any() and torch.isfinite(y).any()
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b.cpu().numpy())
