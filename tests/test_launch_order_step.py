"""Launch-overlap instructions, barriers and bounds checks in the sources of the plan, sparse-attention, norm and sampling
kernels, on the host."""
import os
import re

import pytest

from tests.test_launch_order import CSRC, KERNELS, START, WAIT

FILES = ("attend_chosen.cu", "cache_plan.cu", "cache_select.cu", "norm.cu", "sample.cu")
NEW = [n for n in KERNELS if n.split(":")[0] in FILES]


def test_kernels_are_found():
    assert {n.split(":")[0] for n in NEW} == set(FILES) and len(NEW) >= 8


@pytest.mark.parametrize("name", NEW)
def test_every_kernel_waits_before_dependents_start_and_before_it_leaves(name):
    """Whoever waits for a kernel relies on the ones before it being complete, so no thread leaves before the wait."""
    body = KERNELS[name]
    assert WAIT in body and body.index(WAIT) < body.index(START)
    assert "return" not in re.sub(r"\[[^\]]*\]\([^)]*\)\s*\{[^}]*\}", "", body[: body.index(WAIT)])


def text_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name,access", [
    ("attend_mma.cuh", "table[j >> p.log_p]"), ("attend_mma.cuh", "table[number]"), ("attend_mma.cuh", "cp_async16(dst + L::kK "),
    ("attend_mma.cuh", "cp_async16(dst + L::kKs"), ("attend.cuh", "p.pages[w.s * p.ld_pages + number]"), ("cache_plan.cu", "p.ring[to] ="),
    ("cache_plan.cu", "p.pages + (base + lo)"), ("cache_select.cu", "p.pages[s * p.ld_pages + number]"), ("sample.cu", "p.tokens[row] = index;"),
    ("norm.cu", "store8<VEC>(r, const_cast<void *>(row_of(p.h_out"),
])
def test_accesses_by_device_data_are_checked(name, access):
    """A check stands within the thirty lines before the access, or on its line."""
    text = text_of(name)
    found = list(re.finditer(re.escape(access), text))
    assert found, access
    for m in found:
        before = text[: m.start()].splitlines()[-30:] + [text[m.start():].splitlines()[0]]
        assert any("QMM_DCHECK(" in line for line in before), access
