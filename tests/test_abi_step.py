"""Refusals and size queries of the plan, sparse-attention, norm and sampling calls, on the host: every call fails its
checks (or has nothing to do) before anything is launched."""
import pytest

import block_quantized_matmul_gb300 as qmm

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 1 << 20          # a fake, aligned, non-null address (never dereferenced)
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from block_quantized_matmul_gb300 import build

    build.build()
    return qmm.lib()


def test_plan_refusals(L):
    def f(lens=P, news=P, n_seq=3, P_=16, pages=P, ld=4, ring=P, n_ring=12, at=P, T=5, qs=P, kv=P, slots=P, pos=None, nl=None, na=None):
        return L.qmm_cache_plan(lens, news, n_seq, P_, pages, ld, ring, n_ring, at, T, qs, kv, slots, pos, nl, na, None)

    for bad in ({"n_seq": 0}, {"n_seq": -1}, {"P_": 8}, {"P_": 24}, {"P_": 512}, {"ld": 0}, {"ld": (1 << 27) + 1}, {"n_ring": 0}, {"T": -1},
                {"lens": None}, {"news": None}, {"pages": None}, {"ring": None}, {"at": None}, {"qs": None}, {"kv": None}, {"slots": None}):
        assert f(**bad) == INVALID, bad
    for bad in ({"lens": P + 2}, {"news": P + 1}, {"pages": P + 2}, {"ring": P + 2}, {"at": P + 4}, {"qs": P + 2}, {"kv": P + 1}, {"slots": P + 4},
                {"pos": P + 2}, {"nl": P + 1}, {"na": P + 4}):
        assert f(**bad) == MISALIGNED, bad


def test_sizes(L):
    assert qmm.cache_bounds_size(8, 128) == 8 * 272 and qmm.cache_bounds_size(1, 32) == 80 and qmm.cache_bounds_size(3, 96) == 3 * 208
    assert qmm.cache_bounds_size(2, 256) == 2 * 528 and qmm.cache_bounds_size(1, 64) == 144
    for bad in ((0, 128), (8, 48), (8, 0), (8, 288)):
        assert qmm.cache_bounds_size(*bad) == 0
    assert qmm.cache_select_workspace_size(3, 2, 16, 33) == 256 and qmm.cache_select_workspace_size(100, 8, 64, 65536) == 100 * 8 * 1024 * 4
    for bad in ((0, 2, 16, 33), (3, 0, 16, 33), (3, 2, 24, 33), (3, 2, 16, -1)):
        assert qmm.cache_select_workspace_size(*bad) == 0
    assert qmm.cache_attend_chosen_workspace_size(1, 8, 32, 128, 64, 32) > 0
    assert qmm.cache_attend_chosen_workspace_size(1000, 8, 32, 128, 64, 32) == 0        # enough rows to fill the GPU
    for bad in ((0, 8, 32, 128, 64, 32), (1, 8, 33, 128, 64, 32), (1, 8, 32, 100, 64, 32), (1, 8, 32, 128, 60, 32), (1, 8, 32, 128, 64, 0)):
        assert qmm.cache_attend_chosen_workspace_size(*bad) == 0


CACHE_BAD = ({"H": 0}, {"D": 0}, {"D": 48}, {"D": 288}, {"P_": 8}, {"P_": 24}, {"n_pages": 0}, {"pages": None}, {"qs": None}, {"lens": None}, {"n_seq": 0},
             {"ld": 0}, {"T": -1})


def test_bounds_refusals(L):
    def f(t=1, kc=P, n_pages=4, P_=16, H=2, D=128, pages=P, ld=3, qs=P, lens=P, n_seq=2, T=3, max_new=2, b=P):
        return L.qmm_cache_bounds(t, kc, n_pages, P_, H, D, pages, ld, qs, lens, n_seq, T, max_new, b, None)

    assert f(t=2) == UNSUPPORTED
    for bad in CACHE_BAD + ({"kc": None}, {"b": None}, {"max_new": 0}):
        assert f(**bad) == INVALID, bad
    for bad in ({"kc": P + 8}, {"b": P + 8}, {"pages": P + 2}, {"qs": P + 2}, {"lens": P + 2}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK and f(T=0, b=None, max_new=0) == OK


def test_select_refusals(L):
    need = qmm.cache_select_workspace_size(3, 2, 16, 100)

    def f(b=P, n_pages=4, P_=16, H=2, D=128, pages=P, ld=7, qs=P, lens=P, n_seq=2, dt=BF16, q=P, ldq=512, T=3, Hq=4, tree=None, max_new=2,
          max_len=100, sinks=1, recent=2, budget=4, chosen=P, ws=P, nb=need):
        return L.qmm_cache_select(b, n_pages, P_, H, D, pages, ld, qs, lens, n_seq, dt, q, ldq, T, Hq, tree, max_new, max_len, sinks, recent,
                                  budget, chosen, ws, nb, None)

    assert f(dt=F32) == UNSUPPORTED
    for bad in CACHE_BAD + ({"b": None}, {"q": None}, {"chosen": None}, {"ldq": 504}, {"Hq": 3}, {"Hq": 130, "ldq": 1 << 15}, {"max_new": 0}, {"max_len": -1},
                            {"sinks": -1}, {"recent": 0}, {"budget": 2}, {"budget": 0}, {"budget": 65537}, {"ws": None}, {"nb": need - 1}, {"nb": 0},
                            {"tree": P, "max_new": 65, "budget": 100}, {"tree": P, "budget": 3}):
        assert f(**bad) == INVALID, bad
    for bad in ({"b": P + 8}, {"q": P + 8}, {"ldq": 516}, {"chosen": P + 2}, {"ws": P + 128}, {"tree": P + 4}, {"pages": P + 2}, {"lens": P + 2}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK


def test_attend_chosen_refusals(L):
    def f(t=1, kc=P, vc=P, n_pages=4, P_=16, H=2, D=128, pages=P, ld=3, qs=P, lens=P, n_seq=2, dt=BF16, q=P, ldq=512, T=3, Hq=4, tree=None,
          chosen=P, budget=4, out=P, ldo=512, lse=None, ws=None, nb=0):
        return L.qmm_cache_attend_chosen(t, kc, vc, n_pages, P_, H, D, pages, ld, qs, lens, n_seq, dt, q, ldq, T, Hq, tree, 0.1, chosen, budget,
                                         out, ldo, lse, ws, nb, None)

    assert f(t=3) == UNSUPPORTED and f(dt=F32) == UNSUPPORTED
    for bad in CACHE_BAD + ({"kc": None}, {"vc": None}, {"q": None}, {"out": None}, {"chosen": None}, {"ldq": 504}, {"ldo": 504}, {"Hq": 3}, {"budget": 0},
                            {"budget": 65537}):
        assert f(**bad) == INVALID, bad
    for bad in ({"kc": P + 8}, {"q": P + 8}, {"out": P + 8}, {"ldq": 516}, {"ldo": 516}, {"tree": P + 4}, {"lse": P + 2}, {"chosen": P + 1},
                {"ws": P + 128, "nb": 1 << 20}):
        assert f(**bad) == MISALIGNED, bad
    assert f(T=0) == OK


@pytest.mark.parametrize("form", ["rows", "q8", "mx4"])
def test_norm_refusals(L, form):
    def f(xdt=BF16, x=P, ldx=64, hdt=F32, h=P, ldh=64, R=3, N=64, wp=P, g=P, ldg=64, w=P, ho=P, ldho=64, ydt=F16, y=P, ldy=64, y2=P):
        head = (xdt, x, ldx, hdt, h, ldh, R, N, wp, g, ldg, 1.0, w, 1e-6, ho, ldho)
        if form == "rows":
            return L.qmm_norm(*head, ydt, y, ldy, None)
        return getattr(L, "qmm_norm_" + form)(*head, y, y2, None)

    assert f(xdt=3) == UNSUPPORTED and f(hdt=-1) == UNSUPPORTED
    for bad in ({"R": -1}, {"N": 0}, {"N": 32800, "ldx": 40000, "ldh": 40000, "ldg": 40000, "ldho": 40000, "ldy": 40000}, {"ldx": 63}, {"ldh": 63}, {"ldg": 63},
                {"ldho": 63}, {"h": None}, {"ho": None}, {"y": None}):
        assert f(**bad) == INVALID, bad
    for bad in ({"x": P + 1}, {"h": P + 2}, {"g": P + 1}, {"wp": P + 2}, {"w": P + 1}, {"ho": P + 2}, {"y": P + 1}):
        assert f(**bad) == MISALIGNED, bad
    if form == "rows":
        assert f(ydt=4) == UNSUPPORTED and f(ldy=63) == INVALID
    else:
        assert f(y2=None) == INVALID and f(N=48) == INVALID and f(y=P + 8) == MISALIGNED and f(y2=P + 2) == MISALIGNED
    assert f(R=0) == OK and f(R=0, h=None, y=None, x=None, ho=None) == OK


def test_sample_refusals(L):
    def f(dt=F32, z=P, ld=100, R=2, V=100, t=P, k=P, p=P, q=P, u=P, tok=P, lp=P):
        return L.qmm_sample(dt, z, ld, R, V, t, k, p, q, u, tok, lp, None)

    assert f(dt=3) == UNSUPPORTED
    for bad in ({"R": -1}, {"V": 0}, {"ld": 99}, {"V": (1 << 20) + 1, "ld": 1 << 21}, {"z": None}, {"u": None}, {"tok": None}):
        assert f(**bad) == INVALID, bad
    for bad in ({"z": P + 2}, {"t": P + 2}, {"k": P + 1}, {"p": P + 2}, {"q": P + 2}, {"u": P + 2}, {"tok": P + 2}, {"lp": P + 1}):
        assert f(**bad) == MISALIGNED, bad
    assert f(R=0) == OK and f(R=0, z=None, u=None, tok=None) == OK


def test_binding_raises(L):
    with pytest.raises(qmm.QmmError):
        qmm.qmm_sample("f32", P, 99, 1, 100, None, None, None, None, P, P, None, stream=0)
    with pytest.raises(KeyError):
        qmm.qmm_norm("f64", P, 64, "f32", P, 64, 1, 64, None, None, 0, 1.0, None, 1e-6, P, 64, "f32", P, 64, stream=0)
