"""The debug build's bounds checks, in the sources: every file whose check word qmm_device_status reads has kernels that can
set it, and the accesses whose addresses come from tables or lengths on the device are among what is checked."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_matmul_gb300", "csrc")


def text_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


READERS = [os.path.basename(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "QMM_DCHECK_READER(" in text_of(os.path.basename(p))]


@pytest.mark.parametrize("name", READERS)
def test_a_file_with_a_check_word_has_checks(name):
    assert "QMM_DCHECK(" in text_of(name)


@pytest.mark.parametrize("name,access", [
    ("attend.cu", "table[j >> p.log_p]"), ("attend.cu", "cp_async16(dst + L::kK "), ("attend.cu", "cp_async16(dst + L::kKs"),
    ("attend_tc.cu", "table[j >> p.log_p]"), ("attend_tc.cu", "cp_async16(st + key"), ("attend_tc.cu", "cp_async16(st + L::kRawKs"),
    ("attend.cuh", "p.part_o + part"), ("attend.cuh", "p.pages[w.s * p.ld_pages"), ("cache.cu", "p.pages[s * p.ld_pages"),
    ("cache.cu", "cache + at.codes"), ("mx4_gemm.cu", "bulk_g2s(st + L::kWS"), ("mx4_gemm.cu", "float_to_elem(__uint_as_float(v[c]), y"),
])
def test_accesses_by_device_data_are_checked(name, access):
    """A check stands within the thirty lines before the access."""
    text = text_of(name)
    for m in re.finditer(re.escape(access), text):
        before = text[:m.start()].splitlines()[-30:] + [text[m.start():].splitlines()[0]]
        assert any("QMM_DCHECK(" in line for line in before), access
