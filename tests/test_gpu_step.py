"""The plan, norms, products, sparse attention and sampling together, as a server's steps use them (examples/decode_step.py):
eager steps against plain operations, and the same steps as replays of a graph."""
import importlib.util
import os

import pytest

from tests.gpu_util import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("type_", ["q8_0", "q4_0"])
def test_steps(example, type_):
    lens, tokens = example.main(type_=type_, steps=20)
    assert lens == [90, 23, 53, 120] and len(tokens) == 20 and all(0 <= t < 1000 for row in tokens for t in row)


def test_steps_of_one_request(example):
    lens, tokens = example.main(prompts=(1,), steps=40, seed=5)
    assert lens == [41]


def test_requests_that_come_and_go(example):
    """A request is done and its pages go back, another takes its place, one waits for want of pages: rows of what waits give a
    token all the same, but its length stays."""
    import torch

    s = example.Server(n_pages=14, ld_pages=8, seed=3)
    u = torch.full((4,), 0.3, device="cuda")

    def step(news, max_new):
        rows = sum(max(0, n) for n in news)
        tokens = torch.arange(rows, dtype=torch.int32, device="cuda") % s.vocab
        seen = []
        s.step(tokens, example.int32(news), u, max_new, 128, seen)
        return seen[0]["kv_lens"].tolist(), s.lens.tolist()

    assert step([60, 60, 60, 20], 60) == ([60, 60, 60, 20], [60, 60, 60, 20])          # 4 + 4 + 4 + 2 pages: none is free
    assert step([1, 1, 1, 20], 20) == ([61, 61, 61, 0], [61, 61, 61, 20])              # the last needs a page, and waits
    kv, lens = step([1, -1, 1, 12], 12)                                                # the second is done; 32 tokens fit two pages
    assert kv == [62, 0, 62, 32] and lens == [62, 0, 62, 32]
    assert step([1, 33, 1, 1], 33) == ([63, 33, 63, 33], [63, 33, 63, 33])             # its four pages serve two others
    assert s.ring_at.tolist()[1] - s.ring_at.tolist()[0] == 0
