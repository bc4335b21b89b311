"""MX4 products of more tiles than the GPU has pairs of CTAs: pairs that take two, three and four tiles, with the
accumulator and the ring carried over, in bands of tiles that end ragged, for K of one stage, of fewer stages than the
ring, and of odd numbers of scale blocks."""
import numpy as np
import pytest

from tests.test_gpu_mx4 import check_product, dtypes, operand, torch  # noqa: F401

pytestmark = pytest.mark.gpu


# tiles of 256 x 256: 9 x 12, 3 x 36, 20 x 12, 1 x 77, 80 x 1, 26 x 9 on 76 pairs
@pytest.mark.parametrize("M,N", [(2100, 2900), (600, 9000), (5000, 2900), (100, 19500), (20400, 130), (6500, 2100)])
@pytest.mark.parametrize("K", [32, 256, 384, 1024, 1696])
def test_several_tiles_a_pair(torch, M, N, K):  # noqa: F811
    import block_quantized_matmul_gb300 as qmm

    dtype = {32: "f16", 256: "bf16", 384: "f32", 1024: "bf16", 1696: "f32"}[K]
    ac, as_, a = operand(torch, M, K, seed=M)
    wc, ws, w = operand(torch, N, K, seed=N + 1)
    buf = torch.full((M, N + 3), 7.0, dtype=dtypes(torch)[dtype], device="cuda")
    y = buf[:, :N]
    y.fill_(float("nan"))
    qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, dtype, buf, N + 3)
    check_product(torch, y, a, w, dtype)
    assert (buf[:, N:] == 7).all()


def test_linear_of_several_tiles(torch):  # noqa: F811
    """Rows quantized in the call, then 240 tiles: the same bits as the two calls."""
    import block_quantized_matmul_gb300 as qmm

    M, N, K = 5000, 2900, 800
    wc, ws, _ = operand(torch, N, K, seed=3)
    x = torch.from_numpy(np.random.default_rng(5).standard_normal((M, K)).astype(np.float32)).cuda().to(torch.bfloat16)
    need = qmm.mx4_linear_workspace_size(M, K)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    codes = torch.empty(qmm.mx4_codes_size(M, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(M, K), dtype=torch.uint8, device="cuda")
    for y in outs[:2]:
        qmm.qmm_mx4_linear(wc, ws, K, N, "bf16", x, K, M, "bf16", y, N, wsp, need)
    qmm.qmm_mx4_quantize("bf16", x, M, K, K, codes, scales)
    qmm.qmm_mx4_matmul(wc, ws, K, N, codes, scales, M, "bf16", outs[2], N)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
