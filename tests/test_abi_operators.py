"""Refusals and size queries of the MX4 and cache calls, on the host: every call fails its checks (or has nothing to
do) before anything is launched."""
import pytest

import block_quantized_matmul_gb300 as qmm

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 1 << 20          # a fake, aligned, non-null address (never dereferenced)
BF16 = 2


@pytest.fixture(scope="module")
def L():
    from block_quantized_matmul_gb300 import build

    build.build()
    return qmm.lib()


def test_mx4_sizes(L):
    assert qmm.mx4_codes_size(3, 64) == 96 and qmm.mx4_scales_size(3, 64) == 512
    assert qmm.mx4_scales_size(129, 160) == 2 * 2 * 512 and qmm.mx4_scales_size(14336, 4096) == 112 * 32 * 512
    assert qmm.mx4_codes_size(1 << 31, 1 << 20) == 1 << 50
    for bad in ((0, 64), (-1, 64), (4, 0), (4, 48), (4, 16)):
        assert qmm.mx4_codes_size(*bad) == 0 and qmm.mx4_scales_size(*bad) == 0 and qmm.mx4_linear_workspace_size(*bad) == 0
    assert qmm.mx4_linear_workspace_size(1, 32) == 256 + 512
    assert qmm.mx4_linear_workspace_size(300, 4096) == 300 * 2048 + 3 * 32 * 512


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
def test_mx4_rows_refusals(L, fn):
    def f(dt, x, R, K, ld, codes, scales):
        if fn == "quantize":
            return L.qmm_mx4_quantize(dt, x, R, K, ld, codes, scales, None)
        return L.qmm_mx4_dequantize(codes, scales, R, K, dt, x, ld, None)

    assert f(3, P, 4, 64, 64, P, P) == UNSUPPORTED and f(-1, P, 4, 64, 64, P, P) == UNSUPPORTED
    for R, K, ld in ((0, 64, 64), (-2, 64, 64), (4, 0, 64), (4, 48, 64), (4, 64, 63), ((1 << 31) + 1, 64, 64)):
        assert f(0, P, R, K, ld, P, P) == INVALID
    assert f(0, None, 4, 64, 64, P, P) == INVALID and f(0, P, 4, 64, 64, None, P) == INVALID and f(0, P, 4, 64, 64, P, None) == INVALID
    assert f(0, P + 2, 4, 64, 64, P, P) == MISALIGNED and f(BF16, P + 1, 4, 64, 64, P, P) == MISALIGNED
    assert f(0, P, 4, 64, 64, P + 8, P) == MISALIGNED and f(0, P, 4, 64, 64, P, P + 4) == MISALIGNED


def test_mx4_matmul_refusals(L):
    def f(wc=P, ws=P, K=64, N=32, ac=P, as_=P, M=2, dt=0, y=P, ldy=32):
        return L.qmm_mx4_matmul(wc, ws, K, N, ac, as_, M, dt, y, ldy, None)

    assert f(dt=7) == UNSUPPORTED
    for bad in ({"K": 0}, {"K": 40}, {"N": 0}, {"M": 0}, {"M": -1}, {"ldy": 31}, {"K": 131072 + 32}):
        assert f(**bad) == INVALID, bad
    for name in ("wc", "ws", "ac", "as_", "y"):
        assert f(**{name: None}) == INVALID
    for name in ("wc", "ws", "ac", "as_"):
        assert f(**{name: P + 8}) == MISALIGNED
    assert f(y=P + 2) == MISALIGNED and f(y=P + 1, dt=BF16) == MISALIGNED


def test_mx4_linear_refusals(L):
    need = qmm.mx4_linear_workspace_size(2, 64)

    def f(wc=P, ws=P, K=64, N=32, xdt=0, x=P, ldx=64, M=2, ydt=0, y=P, ldy=32, wsp=P, nb=need):
        return L.qmm_mx4_linear(wc, ws, K, N, xdt, x, ldx, M, ydt, y, ldy, wsp, nb, None)

    assert f(xdt=5) == UNSUPPORTED and f(ydt=5) == UNSUPPORTED
    for bad in ({"K": 40}, {"M": 0}, {"N": -1}, {"ldx": 63}, {"ldy": 31}, {"x": None}, {"wc": None}, {"y": None}, {"wsp": None},
                {"nb": need - 1}, {"nb": 0}):
        assert f(**bad) == INVALID, bad
    assert f(wsp=P + 128) == MISALIGNED and f(x=P + 2) == MISALIGNED and f(ws=P + 1) == MISALIGNED


def test_cache_page_size(L):
    assert qmm.cache_page_size("q8_0", 8, 128, 64) == 8 * 64 * (128 + 8)
    assert qmm.cache_page_size("q4_0", 1, 96, 16) == 16 * (48 + 6)
    for bad in (("iq4_nl", 8, 128, 64), ("q8_0", 0, 128, 64), ("q8_0", 8, 48, 64), ("q8_0", 8, 288, 64), ("q8_0", 8, 0, 64),
                ("q8_0", 8, 128, 8), ("q8_0", 8, 128, 48), ("q8_0", 8, 128, 512), (9, 8, 128, 64)):
        assert qmm.cache_page_size(*bad) == 0, bad


CACHE_BAD = ({"H": 0}, {"D": 0}, {"D": 48}, {"D": 288}, {"P_": 8}, {"P_": 24}, {"P_": 512}, {"n_pages": 0}, {"n_pages": -1}, {"kc": None}, {"vc": None})


def test_cache_write_refusals(L):
    def f(t=1, dt=0, k=P, v=P, ldk=256, ldv=256, T=3, H=2, D=128, slots=P, kc=P, vc=P, n_pages=4, P_=16):
        return L.qmm_cache_write(t, dt, k, v, ldk, ldv, T, H, D, slots, kc, vc, n_pages, P_, None)

    assert f(t=2) == UNSUPPORTED and f(dt=3) == UNSUPPORTED
    for bad in CACHE_BAD + ({"T": -1}, {"ldk": 255}, {"ldv": 0}, {"k": None}, {"v": None}, {"slots": None}):
        assert f(**bad) == INVALID, bad
    for bad in ({"kc": P + 8}, {"vc": P + 8}, {"slots": P + 4}, {"k": P + 2}, {"v": P + 1}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK and f(T=0, k=None, v=None, slots=None) == OK


def test_cache_read_refusals(L):
    def f(t=1, kc=P, vc=P, n_pages=4, P_=16, H=2, D=128, pages=P, ld=3, starts=P, n_seq=2, T=3, dt=0, k=P, v=P, ldk=256, ldv=256):
        return L.qmm_cache_read(t, kc, vc, n_pages, P_, H, D, pages, ld, starts, n_seq, T, dt, k, v, ldk, ldv, None)

    assert f(t=3) == UNSUPPORTED and f(dt=3) == UNSUPPORTED
    for bad in CACHE_BAD + ({"T": -1}, {"ldk": 255}, {"ldv": 0}, {"pages": None}, {"starts": None}, {"n_seq": 0}, {"ld": 0}):
        assert f(**bad) == INVALID, bad
    for bad in ({"kc": P + 8}, {"pages": P + 2}, {"starts": P + 2}, {"k": P + 2}, {"v": P + 1}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK and f(k=None, v=None) == OK


def test_cache_attend_refusals(L):
    def f(t=1, kc=P, vc=P, n_pages=4, P_=16, H=2, D=128, pages=P, ld=3, qs=P, lens=P, n_seq=2, dt=BF16, q=P, ldq=512, T=3, Hq=4,
          tree=None, scale=0.1, max_new=2, max_len=40, out=P, ldo=512, lse=None, ws=None, nb=0):
        return L.qmm_cache_attend(t, kc, vc, n_pages, P_, H, D, pages, ld, qs, lens, n_seq, dt, q, ldq, T, Hq, tree, scale, max_new,
                                  max_len, out, ldo, lse, ws, nb, None)

    assert f(t=3) == UNSUPPORTED and f(dt=0) == UNSUPPORTED and f(dt=3) == UNSUPPORTED
    for bad in CACHE_BAD + ({"T": -1}, {"ldq": 504}, {"ldo": 504}, {"pages": None}, {"qs": None}, {"lens": None}, {"n_seq": 0},
                            {"ld": 0}, {"Hq": 3}, {"Hq": 0}, {"Hq": 130, "ldq": 1 << 15, "ldo": 1 << 15}, {"q": None}, {"out": None},
                            {"max_new": 0}, {"max_len": -1}):
        assert f(**bad) == INVALID, bad
    for bad in ({"kc": P + 8}, {"pages": P + 2}, {"qs": P + 2}, {"lens": P + 1}, {"q": P + 8}, {"out": P + 8}, {"ldq": 516}, {"ldo": 516},
                {"tree": P + 4}, {"lse": P + 2}, {"ws": P + 128, "nb": 1 << 20}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK
    for bad in ((0, 1, 2, 4, 128, 10), (1, 0, 2, 4, 128, 10), (1, 1, 0, 4, 128, 10), (1, 1, 2, 3, 128, 10), (1, 1, 2, 4, 48, 10), (1, 1, 2, 4, 128, -1)):
        assert qmm.cache_attend_workspace_size(*bad) == 0


def test_binding_raises(L):
    with pytest.raises(qmm.QmmError):
        qmm.qmm_mx4_quantize("bf16", P, 1, 48, 48, P, P, stream=0)
    with pytest.raises(KeyError):
        qmm.qmm_mx4_quantize("f64", P, 1, 64, 64, P, P, stream=0)
