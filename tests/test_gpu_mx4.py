"""MX4 operands on the GPU: quantization bit for bit, values exactly, products within their bound, against
plain numpy forms in 64 bits."""
import numpy as np
import pytest

from tests import plain_ops as plain
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


def dtypes(torch):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rows(torch, dtype, R, K, seed, ld=None, offset=0, spread=True):
    """Values of mixed magnitudes in a padded buffer; returns (device view, fp32 values)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, K)).astype(np.float32)
    if spread:
        x *= np.repeat(np.exp2(rng.integers(-6, 7, (R, K // 32))), 32, 1).astype(np.float32)
        x[rng.random((R, K)) < 0.02] = 0
    ld = K if ld is None else ld
    buf = torch.full((offset + R * ld,), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    view = buf[offset:].view(R, ld)
    view[:, :K] = torch.from_numpy(x).cuda().to(dtypes(torch)[dtype])
    return view, view[:, :K].float().cpu().numpy()


def quantize(torch, qmm, dtype, view, R, K, ld):
    codes = torch.full((R, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((qmm.mx4_scales_size(R, K),), 0xFF, dtype=torch.uint8, device="cuda")
    qmm.qmm_mx4_quantize(dtype, view, R, K, ld, codes, scales)
    return codes, scales


def check_operand(codes, scales, x):
    R, K = x.shape
    c, e = plain.mx4_quantize(x)
    got = scales.cpu().numpy()
    np.testing.assert_array_equal(got[plain.mx4_scale_index(R, K)], e)
    K4 = -(-K // 128) * 128
    pad = plain.mx4_scale_index(R, K4)[:, K // 32:]
    assert (got[pad] == 0).all()
    np.testing.assert_array_equal(codes.cpu().numpy(), plain.mx4_pack_codes(c))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,K,ld,offset", [(1, 32, 32, 0), (3, 64, 64, 0), (128, 128, 128, 0), (129, 160, 160, 0), (5, 4096, 4096, 0),
                                           (7, 288, 296, 8), (7, 288, 291, 1), (300, 1056, 1056, 0)])
def test_quantize_bit_exact(torch, dtype, R, K, ld, offset):
    import block_quantized_matmul_gb300 as qmm

    view, x = rows(torch, dtype, R, K, seed=R * K, ld=ld, offset=offset)
    check_operand(*quantize(torch, qmm, dtype, view, R, K, ld), x)


def test_quantize_special_values(torch):
    import block_quantized_matmul_gb300 as qmm

    f = np.float32
    x = np.zeros((12, 64), f)
    x[1, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0]                # ties, scale 1
    x[2, :8] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -7.9]
    x[3, 0], x[3, 40] = np.finfo(f).max, -np.finfo(f).max                   # saturates at 6 * 2^125
    x[4, :4] = [1e-45, -3e-45, 1e-40, 1e-39]                                # subnormal largest: scale 2^-127
    x[5, 3], x[6, 35], x[7, 5], x[7, 6] = np.nan, np.inf, -np.inf, 3.0      # whole blocks are NaN
    x[8, :3] = [-0.0, 0.0, -1e-3]
    x[8, 3] = 6.0
    x[9, :2] = [np.float32(2.0 ** -125), 2.0 ** -126]                       # exponents at the scale's lower end
    x[10] = np.linspace(-8, 8, 64)
    x[11] = np.float32(2.0) ** np.arange(-32, 32)
    view = torch.from_numpy(x).cuda()
    codes, scales = quantize(torch, qmm, "f32", view, 12, 64, 64)
    check_operand(codes, scales, x)
    y = torch.empty(12, 64, device="cuda")
    qmm.qmm_mx4_dequantize(codes, scales, 12, 64, "f32", y, 64)
    np.testing.assert_array_equal(y.cpu().numpy(), plain.mx4_values(*plain.mx4_quantize(x)).astype(f))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,K,ld,offset", [(1, 32, 32, 0), (130, 416, 416, 0), (6, 96, 99, 3)])
def test_dequantize_exact(torch, dtype, R, K, ld, offset):
    import block_quantized_matmul_gb300 as qmm

    rng = np.random.default_rng(R)
    c = rng.integers(0, 16, (R, K), dtype=np.uint8)
    e = rng.integers(127 - 12, 127 + 12, (R, K // 32)).astype(np.uint8)
    buf = torch.full((offset + R * ld,), -7.0, dtype=dtypes(torch)[dtype], device="cuda")
    y = buf[offset:].view(R, ld)
    qmm.qmm_mx4_dequantize(torch.from_numpy(plain.mx4_pack_codes(c)).cuda(), torch.from_numpy(plain.mx4_pack_scales(e, K, 0xFF)).cuda(),
                           R, K, dtype, y, ld)
    want = torch.from_numpy(plain.mx4_values(c, e)).to(dtypes(torch)[dtype])
    assert torch.equal(y[:, :K].cpu().float(), want.float())
    assert (buf[:offset] == -7).all() and (y[:, K:] == -7).all()


def operand(torch, R, K, seed, lo=-3, hi=4, positive=False):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 8 if positive else 16, (R, K), dtype=np.uint8)
    e = rng.integers(127 + lo, 127 + hi, (R, K // 32)).astype(np.uint8)
    return (torch.from_numpy(plain.mx4_pack_codes(c)).cuda(), torch.from_numpy(plain.mx4_pack_scales(e, K, 0xFF)).cuda(),
            plain.mx4_values(c, e))


def reference(torch, a, w):
    """fp64 products on the GPU (plain matrix product): (sum, sum of magnitudes)."""
    a, w = torch.from_numpy(a).cuda(), torch.from_numpy(w).cuda()
    return a @ w.t(), a.abs() @ w.abs().t()


def check_product(torch, y, a, w, dtype):
    ref, mag = reference(torch, a, w)
    # the stated bound of the fp32 sum, and one rounding to the output's type (fp16: or half its smallest step)
    tol = 1e-5 * mag + plain.ULP[dtype] * (ref.abs() + 1e-5 * mag) + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = (y.double() - ref).abs()
    top = {"f32": 3.4e38, "f16": 65504.0, "bf16": 3.38e38}[dtype]
    fine = (err <= tol) | (ref.abs() > top * 0.999) & torch.isinf(y)
    assert fine.all(), (int((~fine).sum()), float(err.max()))


SHAPES = [(1, 32, 1), (1, 64, 5), (1, 4096, 4096), (2, 96, 130), (8, 256, 128), (9, 288, 257), (16, 512, 384), (17, 544, 100),
          (33, 1056, 300), (64, 2048, 129), (100, 160, 1000), (128, 128, 128), (200, 1024, 515), (255, 416, 640), (513, 768, 900)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_matmul(torch, M, K, N, dtype):
    import block_quantized_matmul_gb300 as qmm

    ac, as_, a = operand(torch, M, K, seed=M + K)
    wc, ws, w = operand(torch, N, K, seed=N + K + 1)
    y = torch.full((M, N), float("nan"), dtype=dtypes(torch)[dtype], device="cuda")
    qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, dtype, y, N)
    check_product(torch, y, a, w, dtype)


@pytest.mark.parametrize("M,K,N", [(1, 14336, 300), (40, 8192, 260), (130, 16384, 140)])
def test_matmul_long_rows_of_one_sign(torch, M, K, N):
    """All products positive: every partial sum grows, the worst case for the fp32 sums."""
    import block_quantized_matmul_gb300 as qmm

    ac, as_, a = operand(torch, M, K, seed=1, lo=0, hi=1, positive=True)
    wc, ws, w = operand(torch, N, K, seed=2, lo=-5, hi=6, positive=True)
    y = torch.empty(M, N, device="cuda")
    qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, "f32", y, N)
    check_product(torch, y, a, w, "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_matmul_output_stride(torch, M, dtype):
    import block_quantized_matmul_gb300 as qmm

    K, N, ld = 256, 133, 150
    ac, as_, a = operand(torch, M, K, seed=3)
    wc, ws, w = operand(torch, N, K, seed=4)
    buf = torch.full((1 + M * ld,), 7.0, dtype=dtypes(torch)[dtype], device="cuda")
    y = buf[1:].view(M, ld)
    qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, dtype, y, ld)
    check_product(torch, y[:, :N], a, w, dtype)
    assert buf[0] == 7 and (y[:, N:] == 7).all()


@pytest.mark.parametrize("M", [1, 30, 300])
def test_matmul_nan_scales_and_padding(torch, M):
    """A NaN block makes its own row's results NaN and no others; what rows past R hold in the scales does not matter."""
    import block_quantized_matmul_gb300 as qmm

    K, N = 160, 200
    rng = np.random.default_rng(7)
    c, e = rng.integers(0, 16, (N, K), dtype=np.uint8), rng.integers(120, 130, (N, K // 32)).astype(np.uint8)
    e[11, 4], e[150, 0] = 255, 255
    wc, ws = torch.from_numpy(plain.mx4_pack_codes(c)).cuda(), torch.from_numpy(plain.mx4_pack_scales(e, K, 0xFF)).cuda()
    ac, as_, a = operand(torch, M, K, seed=8)
    y = torch.empty(M, N, device="cuda")
    qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, "f32", y, N)
    nan = torch.isnan(y)
    assert nan[:, [11, 150]].all() and nan.sum() == 2 * M
    keep = np.setdiff1d(np.arange(N), [11, 150])
    check_product(torch, y[:, torch.from_numpy(keep).cuda()], a, plain.mx4_values(c, e)[keep], "f32")


def test_matmul_scale_range(torch):
    """Scales far from 1 on both sides: the whole E8M0 range is kept as long as the products are fp32 numbers."""
    import block_quantized_matmul_gb300 as qmm

    K, N, M = 64, 128, 4
    for wa, aa in ((-100, 90), (100, -95), (-120, 120), (60, 40)):
        wc, ws, w = operand(torch, N, K, seed=5, lo=wa, hi=wa + 3)
        ac, as_, a = operand(torch, M, K, seed=6, lo=aa, hi=aa + 3)
        y = torch.empty(M, N, device="cuda")
        qmm.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, "f32", y, N)
        check_product(torch, y, a, w, "f32")


@pytest.mark.parametrize("xdt,ydt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("M,K,N", [(1, 512, 260), (5, 1056, 129), (70, 288, 1000), (140, 4096, 256)])
def test_linear_is_quantize_and_matmul(torch, M, K, N, xdt, ydt):
    import block_quantized_matmul_gb300 as qmm

    view, x = rows(torch, xdt, M, K, seed=M, ld=K + 8)
    wc, ws, w = operand(torch, N, K, seed=9)
    need = qmm.mx4_linear_workspace_size(M, K)
    wsp = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    at = wsp.data_ptr() + (-wsp.data_ptr()) % 256
    y = torch.empty(M, N, dtype=dtypes(torch)[ydt], device="cuda")
    qmm.qmm_mx4_linear(wc, ws, K, N, xdt, view, K + 8, M, ydt, y, N, at, need)
    codes, scales = quantize(torch, qmm, xdt, view, M, K, K + 8)
    y2 = torch.empty_like(y)
    qmm.qmm_mx4_matmul(wc, ws, K, N, codes, scales, M, ydt, y2, N)
    assert torch.equal(y, y2)
    check_product(torch, y, plain.mx4_values(*plain.mx4_quantize(x)), w, ydt)


def test_repeatable_and_on_other_streams(torch):
    import block_quantized_matmul_gb300 as qmm

    outs = []
    wc, ws, w = operand(torch, 700, 2048, seed=10)
    view, x = rows(torch, "bf16", 60, 2048, seed=11)
    torch.cuda.synchronize()
    for i in range(6):
        s = torch.cuda.Stream()
        need = qmm.mx4_linear_workspace_size(60, 2048)
        with torch.cuda.stream(s):
            wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
            y = torch.full((60, 700), float("nan"), device="cuda")
            qmm.qmm_mx4_linear(wc, ws, 2048, 700, "bf16", view, 2048, 60, "f32", y, 700, wsp, need, stream=s if i % 2 else None)
        outs.append((y, wsp, s))
    torch.cuda.synchronize()
    for y, _, _ in outs[1:]:
        assert torch.equal(y, outs[0][0])
    check_product(torch, outs[0][0], plain.mx4_values(*plain.mx4_quantize(x)), w, "f32")


def test_captured_in_a_graph(torch):
    import block_quantized_matmul_gb300 as qmm

    wc, ws, w = operand(torch, 300, 1024, seed=12)
    view, x = rows(torch, "bf16", 3, 1024, seed=13)
    need = qmm.mx4_linear_workspace_size(3, 1024)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    y = torch.zeros(3, 300, device="cuda")
    call = lambda: qmm.qmm_mx4_linear(wc, ws, 1024, 300, "bf16", view, 1024, 3, "f32", y, 300, wsp, need)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    first = y.clone()
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)
    check_product(torch, y, plain.mx4_values(*plain.mx4_quantize(x)), w, "f32")
