"""A product queued directly behind an attention of many rows (tcgen05, not split), whose CTAs may share an SM: results as
with a synchronization in between."""
import numpy as np
import pytest

from tests.gpu_util import torch_mod
from tests.test_gpu_cache import Case, device

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
@pytest.mark.parametrize("new,G,D", [(4, 16, 64), (3, 12, 32), (4, 16, 128)])
def test_product_behind_attention(torch, type_, new, G, D):
    import block_quantized_matmul_gb300 as qmm

    lens = [700, 90]
    c = Case(torch, type_, lens, 2, D, 16).upload()
    T, Hq, width, n = new, 2 * G, 2 * G * D, 2000
    rng = np.random.default_rng(0)
    q = device(torch, rng.standard_normal((T, width)).astype(np.float32)).to(torch.bfloat16)
    w = device(torch, rng.standard_normal((n, width)).astype(np.float32))
    codes = torch.empty(qmm.mx4_codes_size(n, width), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qmm.mx4_scales_size(n, width), dtype=torch.uint8, device="cuda")
    qmm.qmm_mx4_quantize("f32", w, n, width, width, codes, scales)
    need = qmm.mx4_linear_workspace_size(T, width)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    starts, kv = (device(torch, np.array(v, np.int32)) for v in ([0, new, new], lens))
    runs = []
    for i in range(20):
        o = torch.empty_like(q)
        y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
        qmm.qmm_cache_attend(type_, c.k_cache, c.v_cache, c.n_pages, 16, 2, D, c.pages, c.table.shape[1], starts, kv, 2, "bf16", q, width, T, Hq,
                             None, 0.1, new, max(lens), o, width, None, None, 0)
        if i == 0:
            torch.cuda.synchronize()
        qmm.qmm_mx4_linear(codes, scales, width, n, "bf16", o, width, T, "bf16", y, n, ws, need)
        # and a product of ready operands directly behind the attention: 20 rows of the weight as activations
        qmm.qmm_cache_attend(type_, c.k_cache, c.v_cache, c.n_pages, 16, 2, D, c.pages, c.table.shape[1], starts, kv, 2, "bf16", q, width, T, Hq,
                             None, 0.1, new, max(lens), o, width, None, None, 0)
        z = torch.empty(20, n, device="cuda")
        qmm.qmm_mx4_matmul(codes, scales, width, n, codes, scales, 20, "f32", z, n)
        runs.append((o, y, z))
    torch.cuda.synchronize()
    for run in runs[1:]:
        for a, b in zip(run, runs[0]):
            assert torch.equal(a, b)
    assert torch.isfinite(runs[0][1]).all()
