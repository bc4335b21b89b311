"""MX4 products with long rows of one sign, in every kernel: the stated bound, 1e-5 of the sum of magnitudes, holds for every K
that the calls take.  The tensor cores round sums towards zero, so with data of one sign the error grows with the
products that one accumulator takes (4.5e-5 at K = 131072 in a single one)."""
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


class Operand:
    """Random codes (of one sign, or both) with scales 2^-5 to 2^5, made on the GPU."""

    def __init__(self, torch, R, K, seed, signs):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.R, self.K = torch, R, K
        byte = torch.randint(0, 256, (R, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        self.codes = byte if signs else byte & 0x77
        self.e = torch.randint(122, 133, (R, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
        n128 = -(-K // 128)
        self.scales = torch.zeros(-(-R // 128) * n128 * 512, dtype=torch.uint8, device="cuda")
        b = torch.arange(K // 32, device="cuda")[None]
        for r0 in range(0, R, 1024):
            r = torch.arange(r0, min(R, r0 + 1024), device="cuda")[:, None]
            self.scales[(r // 128 * n128 + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = self.e[r0:r0 + 1024]

    def values(self, r0, r1):
        t = self.torch
        table = t.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=t.float64, device="cuda")
        c = self.codes[r0:r1]
        v = table[t.stack((c & 15, c >> 4), -1).int()].view(c.shape[0], -1, 32)
        return (v * t.pow(2.0, self.e[r0:r1].double() - 127)[..., None]).view(c.shape[0], -1)


@pytest.mark.parametrize("signs", [False, True], ids=["one_sign", "both_signs"])
@pytest.mark.parametrize("M,N,K", [
    (4, 256, 131072), (32, 130, 65568),                        # few tokens, K shared by a cluster
    (3, 19700, 131072), (20, 19700, 28672), (32, 19600, 131072),   # few tokens, a CTA takes all of K
    (1, 300, 28672), (33, 257, 16416), (64, 256, 131072), (300, 520, 33024),   # 16416: one stage past the first accumulator
    (600, 9000, 20000),                                        # pairs that take several tiles
])
def test_bound_holds_for_long_rows(torch, M, N, K, signs):
    import block_quantized_matmul_gb300 as qmm

    a, w = Operand(torch, M, K, 1, signs), Operand(torch, N, K, 2, signs)
    y = torch.full((M, N), float("nan"), device="cuda")
    qmm.qmm_mx4_matmul(w.codes, w.scales, K, N, a.codes, a.scales, M, "f32", y, N)
    again = torch.full((M, N), float("nan"), device="cuda")
    qmm.qmm_mx4_matmul(w.codes, w.scales, K, N, a.codes, a.scales, M, "f32", again, N)
    assert torch.equal(y, again)
    av = a.values(0, M)
    for n0 in range(0, N, 2048):
        wv = w.values(n0, min(N, n0 + 2048))
        ref, mag = av @ wv.t(), av.abs() @ wv.abs().t()
        err = (y[:, n0:n0 + 2048].double() - ref).abs()
        # the bound of the fp32 sum, and one rounding to fp32
        assert (err <= 1e-5 * mag + 2.0 ** -24 * ref.abs()).all(), float((err / mag).max())


@pytest.mark.parametrize("M", [2, 40])
def test_linear_is_quantize_and_matmul_for_long_rows(torch, M):
    import block_quantized_matmul_gb300 as qmm

    K, N = 40000, 300
    w = Operand(torch, N, K, 3, True)
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.bfloat16)
    need = qmm.mx4_linear_workspace_size(M, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y, y2 = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    qmm.qmm_mx4_linear(w.codes, w.scales, K, N, "bf16", x, K, M, "f32", y, N, ws, need)
    codes = torch.empty(qmm.mx4_codes_size(M, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(M, K), dtype=torch.uint8, device="cuda")
    qmm.qmm_mx4_quantize("bf16", x, M, K, K, codes, scales)
    qmm.qmm_mx4_matmul(w.codes, w.scales, K, N, codes, scales, M, "f32", y2, N)
    assert torch.equal(y, y2)
