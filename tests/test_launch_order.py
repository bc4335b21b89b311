"""The order of launch-overlap instructions in the kernels' sources, on the host: what a GPU test could only show by
hanging, or by a race that it may not meet."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_matmul_gb300", "csrc")
START, WAIT, ALLOC = "griddepcontrol.launch_dependents", "griddepcontrol.wait", "tcgen05.alloc"


def kernels():
    """{name: body without comments} of every __global__ function of the library."""
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            name = re.search(r"(\w+_kernel)\s*\(", text[m.end():])
            at = text.index("{", m.end() + name.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            found[f"{os.path.basename(path)}:{name.group(1)}"] = text[at:end]
    return found


KERNELS = kernels()


def test_kernels_are_found():
    assert len(KERNELS) >= 20 and "attend_tc.cu:attend_tc_kernel" in KERNELS and "mx4_gemm.cu:mx4_pair_kernel" in KERNELS


@pytest.mark.parametrize("name", [n for n, body in KERNELS.items() if ALLOC in body and START in body])
def test_tensor_memory_is_allocated_before_dependents_start(name):
    """A dependent that allocates tensor memory and then waits for this kernel must not be able to take the columns that
    a CTA of this kernel still has to allocate: neither could go on."""
    body = KERNELS[name]
    assert body.index(ALLOC) < body.index(START)
    assert "__syncthreads" in body[body.index(ALLOC):body.index(START)] or "barrier.cluster.wait" in body[body.index(ALLOC):body.index(START)]


@pytest.mark.parametrize("name", ["repack.cu:repack_kernel", "repack.cu:repack_q4k_kernel", "mx4.cu:mx4_quantize_kernel"])
def test_weights_are_visible_when_their_kernel_exits(name):
    """Kernels that stream a weight before they wait rely on it: a fence behind the last store."""
    body = KERNELS[name]
    last_store = max(m.start() for m in re.finditer(r"[^=!<>]=[^=]", body))
    assert "__threadfence()" in body[last_store:]


@pytest.mark.parametrize("name", [n for n, body in KERNELS.items() if START in body and n.startswith(("mx4", "cache", "attend."))
                                  or n.startswith("attend_tc")])
def test_dependents_start_after_the_wait(name):
    """A kernel that reads its weight before it waits relies on the one before it: that has seen everything before itself
    complete when it lets others start.  The join starts them sooner, behind an attention that has waited."""
    body = KERNELS[name]
    if name == "attend.cu:attend_join_kernel":
        assert all(KERNELS[n].index(WAIT) < KERNELS[n].index(START) for n in ("attend.cu:attend_kernel", "attend_tc.cu:attend_tc_kernel"))
    else:
        assert body.index(WAIT) < body.index(START)


@pytest.mark.parametrize("name", ["mx4_gemm.cu:mx4_gemm_kernel", "mx4_gemm.cu:mx4_pair_kernel"])
def test_bounded_waits_start_after_the_wait(name):
    """A wait with a limit must not have the kernel before in it, which may take any time: each warp's part waits for that
    kernel (without a limit) before its first bounded wait."""
    body = KERNELS[name]
    roles = re.split(r"if \(warp == 0\) \{|\} else if \(warp == 1\) \{\s*\n|\n    \} else \{", body[body.rindex("uint32_t tmem = *tmem_slot"):])[1:4]
    assert len(roles) == 3
    for part in roles:
        first = re.search(r"wait_(bounded|warp|cluster_bounded)\(", part)
        assert first and WAIT in part[:first.start()]
