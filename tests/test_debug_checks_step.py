"""The debug build's bounds checks of the plan, sparse-attention, norm and sampling kernels, in the sources: each access whose place
comes from data on the device stands behind a check of that very place, in the statement itself or in a condition that encloses it or
leaves before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_matmul_gb300", "csrc")

# file, the access, and what has to be checked before it
CHECKED = [
    ("attend_mma.cuh", "w.list[j >> p.log_p]", "(j >> p.log_p) < p.list_len"),
    ("attend_mma.cuh", "half.page = table[number]", "number < p.ld_pages"),
    ("attend_mma.cuh", "half.page = table[j >> p.log_p]", "(j >> p.log_p) < p.ld_pages"),
    ("attend_mma.cuh", "cp_async16(dst + L::kK ", "src >= 0 && src + 16 <= p.n_pages * page_bytes"),
    ("attend_mma.cuh", "cp_async16(dst + L::kV ", "src >= 0 && src + 16 <= p.n_pages * page_bytes"),
    ("attend_mma.cuh", "cp_async16(dst + L::kKs", "src >= 0 && src + 16 <= p.n_pages * page_bytes"),
    ("attend_mma.cuh", "cp_async16(dst + L::kVs", "src >= 0 && src + 16 <= p.n_pages * page_bytes"),
    ("attend.cuh", "number = w.list[number]", "number < p.list_len"),
    ("attend.cuh", "p.pages[w.s * p.ld_pages + number]", "number < p.ld_pages && w.s < p.n_seq"),
    ("attend.cuh", "p.part_ml[2 * part] = top", "row < w.rows && w.q0 + i < p.T && hq < Hq && d + N <= D && w.sp < w.used && (w.used == 1 || w.used <= p.splits)"),
    ("attend_chosen.cu", "join_row<DB, WPR>(p, at, tok, hq, used)", "used <= p.splits"),
    ("cache_plan.cu", "page[u] = p.pages[(base + lo) * p.ld_pages + k]", "k < p.ld_pages && base + lo < p.n_seq"),
    ("cache_plan.cu", "p.ring[to] = page[u]", "to >= 0 && to < p.n_ring"),
    ("cache_plan.cu", "p.pages + (base + lo) * p.ld_pages + number", "number < p.ld_pages && base + lo < p.n_seq"),
    ("cache_select.cu", "p.pages[s * p.ld_pages + number]", "number < p.ld_pages"),
    ("cache_select.cu", "out[number] = there[e]", "number < p.most && number < p.ld_pages"),
    ("cache_select.cu", "few[to] = key", "to < kFew"),
    ("sample.cu", "p.tokens[row] = index;", "index >= 0 && index < p.V"),
    ("norm.cu", "store8<VEC>(r, const_cast<void *>(row_of(p.h_out", "!VEC || at + 8 <= n"),
]


def block_end(text, at):
    """Where the block that `at` lies in ends."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth < 0:
            return i
    return len(text)


def guarded(text, start, end):
    """(from, to): what a check at text[start:end] keeps from running when it fails: the statement or block of its `if`, or, where a failed
    check leaves, all that follows in its block."""
    leaves = re.match(r"\)+\s*(return|continue)\b", text[end:])
    if text[start - 1] == "!":
        return (end, block_end(text, end)) if leaves else (end, end)
    body = re.match(r"\)+\s*", text[end:])
    at = end + (body.end() if body else 0)
    return (at, block_end(text, at + 1)) if text[at] == "{" else (at, text.index(";", at) + 1)


@pytest.mark.parametrize("name,access,check", CHECKED, ids=[f"{n}:{a[:24]}" for n, a, _ in CHECKED])
def test_the_place_of_an_access_is_checked(name, access, check):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = list(re.finditer(re.escape(access), text))
    assert found, access
    for m in found:
        spans = [guarded(text, c.start(), c.end()) for c in re.finditer(re.escape(f"QMM_DCHECK({check})"), text[: m.start()])]
        assert any(a <= m.start() < b for a, b in spans), (access, check)


@pytest.mark.parametrize("text,fine", [
    ("{ if (QMM_DCHECK(i < n)) a[i] = 0; }", True), ("{ if (x && QMM_DCHECK(i < n)) { y(); a[i] = 0; } }", True),
    ("{ if (!QMM_DCHECK(i < n)) return; a[i] = 0; }", True), ("{ { if (!QMM_DCHECK(i < n)) return; } a[i] = 0; }", False),
    ("{ if (QMM_DCHECK(i < n)) y(); a[i] = 0; }", False), ("{ (void)!QMM_DCHECK(i < n); a[i] = 0; }", False), ("{ if (QMM_DCHECK(i < n)) { y(); } a[i] = 0; }", False),
])
def test_what_a_check_guards(text, fine):
    c = re.search(r"QMM_DCHECK\(i < n\)", text)
    a, b = guarded(text, c.start(), c.end())
    assert (a <= text.index("a[i]") < b) == fine
