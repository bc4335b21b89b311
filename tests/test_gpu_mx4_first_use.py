"""An MX4 weight that is used by the call right after the one that quantized it, again and again in the same buffers: every
product is that of the new weight."""
import pytest

from tests.gpu_util import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    return t


@pytest.mark.parametrize("M", [1, 4, 9])
@pytest.mark.parametrize("N,K", [(300, 512), (4096, 4096)])
def test_product_right_after_quantization(torch, M, N, K):
    import block_quantized_matmul_gb300 as qmm

    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    weights = [torch.randn(N, K, generator=gen, device="cuda") for _ in range(4)]
    codes = torch.empty(qmm.mx4_codes_size(N, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(N, K), dtype=torch.uint8, device="cuda")
    need = qmm.mx4_linear_workspace_size(M, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def product(w, y, wait):
        qmm.qmm_mx4_quantize("f32", w, N, K, K, codes, scales)
        if wait:
            torch.cuda.synchronize()
        qmm.qmm_mx4_linear(codes, scales, K, N, "bf16", x, K, M, "f32", y, N, ws, need)

    want = [torch.empty(M, N, device="cuda") for _ in weights]
    for w, y in zip(weights, want):
        product(w, y, True)
        torch.cuda.synchronize()
    got = [torch.full((M, N), float("nan"), device="cuda") for _ in range(40)]
    for i, y in enumerate(got):
        product(weights[i % 4], y, False)
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i
