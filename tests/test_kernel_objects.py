"""What the built library's kernels take of a CU, and which of them there are
(no GPU: read from the code objects)."""
import pytest

from few_row_quantized_amd import qgemv as q

from kernel_objects import kernels


@pytest.fixture(scope="module")
def all_kernels():
    found = kernels(q.LIB_PATH)
    assert len(found) > 300
    return found


def test_no_kernel_has_more_than_64_kib_of_lds_of_its_own(all_kernels):
    """More is asked for at the launch (dynamic LDS), after the runtime has
    allowed it for the kernel."""
    more = {k: d[".group_segment_fixed_size"] for k, d in all_kernels.items()
            if d[".group_segment_fixed_size"] > 64 * 1024}
    assert not more
