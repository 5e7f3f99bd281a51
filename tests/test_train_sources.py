"""Properties of the training kernels' sources that a run cannot show reliably:
what happens between the threads of a warp depends on how they are scheduled."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verify_ssd_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name,kernels", [("ssd_rows.cuh", 2), ("ssd_linear.cuh", 1)])
def test_barriers_are_published_before_they_are_polled(name, kernels):
    """Between a thread's initialisation of an mbarrier and the next use of one,
    all threads that may poll it meet at a barrier."""
    body = source(name)
    starts = [m.end() for m in re.finditer(r"mbar_init_fence\(\);", body)]
    assert len(starts) == kernels
    for at in starts:
        use = re.search(r"\b(slice_load|slice_wait|mbar_wait_bounded|mbar_try_wait|wait)\(", body[at:])
        assert re.search(r"__syncwarp\(\)|__syncthreads\(\)|\.sync\(\)", body[at:at + use.start()]), body[at:at + use.end()]


def test_a_warp_gives_up_as_one():
    """A wait that a whole warp takes ends it for all lanes or for none; the
    other waits of the product kernel are one lane's."""
    body = source("ssd_linear.cuh")
    kernel = body[body.index("ssd_gemm_kernel(const"):]
    epilogue = kernel[kernel.index("const int quad"):kernel.index("ssd_linear_prep_kernel")]
    waits = re.findall(r"[^;\n]*\bwait\(&[^;\n]*", epilogue)
    assert len(waits) == 1 and "__all_sync(0xFFFFFFFFu, wait(" in waits[0]


def test_a_cluster_part_is_late_for_a_warp_as_one():
    """All lanes of the joining warp share one verdict on the cluster's parts,
    and a block that gave up alone leaves NaN, not zeros, in its slice."""
    body = source("ssd_rows.cuh")
    kernel = body[body.index("ssd_distill_kernel(const"):]
    waits = re.findall(r"[^;\n]*\bparts_wait\(&[^;\n]*", kernel)
    assert len(waits) == 1 and "__reduce_or_sync(0xFFFFFFFFu" in waits[0]
    assert re.search(r"j\.late \? 0x7FC07FC0u : 0u", kernel)
