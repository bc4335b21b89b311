"""How the attention over the block-quantized cache cuts a batch's sequences into splits, restated on the host from
csrc/attend.cu (split_of) and csrc/attend.cuh (fewest_steps, chunk_of), 32-bit arithmetic included: whatever the lengths
are, empty sequences among them, there is a CTA for every split and room in the workspace for its result."""
import random

import pytest

STEP, M32 = 128, 0xFFFFFFFF


def up_div(a, b):
    return -(-a // b)


def split_of(n_seq, H, row_tiles, tcgen05, max_len):
    places, per = (152 if tcgen05 else 304), H * row_tiles
    s = {"splits": 1, "budget": n_seq, "waves": 1, "fixed": 2 if tcgen05 else 6}
    if n_seq * per >= places:
        return s
    s["budget"], s["waves"] = places // per, 2 if 2 * n_seq * per > places else 1
    every = s["budget"] * s["waves"]
    s["splits"] = max(1, min(every - n_seq + 1, 4 * up_div(every, n_seq), up_div(max_len, STEP)))
    return s


def count(steps, c):
    """Splits of sequences of so many steps, c steps to a split, as a lane counts them."""
    inv, up = (M32 // c + (c > 1)) & M32, max(c - 1, 1)
    return sum(max(1, (((t + up) & M32) * inv) >> 32) for t in steps)


def fewest_steps(steps, s, budget):
    most = max(steps)
    lo = max(1, up_div(most, s["splits"]), up_div(sum(steps) & M32, budget))
    hi = max(lo, most)
    for _ in range(2):
        if lo >= hi:
            break
        sizes = [lo + (hi - lo) * lane // 31 for lane in range(32)]
        fits = [count(steps, c) <= budget for c in sizes]
        first = fits.index(True) if True in fits else -1
        hi = sizes[first]
        if first == 0:
            break
        lo = sizes[first - 1] + 1
    return hi


def chunk_of(steps, s):
    if len(steps) == 1:
        return max(1, up_div(steps[0], s["splits"]), up_div(steps[0], s["budget"]))
    c = fewest_steps(steps, s, s["budget"])
    if s["waves"] == 2:
        c2 = fewest_steps(steps, s, 2 * s["budget"])
        if 2 * (c2 + s["fixed"]) < c + s["fixed"]:
            c = c2
    return c


def check(lens, H, row_tiles, tcgen05, max_len):
    s = split_of(len(lens), H, row_tiles, tcgen05, max_len)
    if s["splits"] < 2:
        return
    steps = [up_div(n, STEP) for n in lens]
    c = chunk_of(steps, s)
    used = [max(1, up_div(t, c)) for t in steps]
    assert sum(used) <= s["budget"] * s["waves"], (lens, s, c)
    assert max(used) <= s["splits"], (lens, s, c)


@pytest.mark.parametrize("c", [1, 2, 3, 5, 31, 32, 1000, 46340])
def test_count_is_the_division_rounded_up(c):
    rng = random.Random(c)
    for t in [0, 1, 2, c - 1, c, c + 1, 2 * c, 46340] + [rng.randrange(0, 46341) for _ in range(500)]:
        assert count([t], c) == max(1, up_div(t, c)), t


@pytest.mark.parametrize("lens,H", [([433, 0, 1904], 16), ([0, 500] * 8, 8), ([0, 512, 512, 1024] + [256] * 11, 8),
                                    ([0] * 9 + [384] * 2 + [512] * 8, 8)])
def test_empty_sequences(lens, H):
    check(lens, H, 1, False, 4096)


@pytest.mark.parametrize("seed", range(4))
def test_random_batches(seed):
    rng = random.Random(seed)
    for _ in range(4000):
        empty, top = rng.choice([0, 0.3, 0.6]), rng.choice([300, 1000, 5000, 70000, 2 ** 27])
        lens = [0 if rng.random() < empty else rng.randrange(0, top) for _ in range(rng.randrange(1, 40))]
        check(lens, rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 3]), rng.random() < 0.5, max(max(lens), rng.choice([1, 4096, 100000])))
