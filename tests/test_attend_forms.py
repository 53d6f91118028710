"""The attention's kernels in the built library against the plan (no GPU)."""
import pytest

from few_row_quantized_amd import qgemv as q

from kernel_config import attend_form
from kernel_objects import instances


@pytest.mark.parametrize("after_prefix", [False, True])
def test_the_library_has_the_kernels_that_calls_reach_and_no_others(after_prefix):
    want = {(bf, f8, dim, tiles, split)
            for bf in (0, 1) for f8 in (0, 1) for dim in (64, 128, 256)
            for split, tiles in {attend_form(rows, dim, bool(f8), short, after_prefix)
                                 for rows in range(1, q.MAX_M * q.MAX_GROUP + 1) for short in (False, True)}}
    # the last two: workgroups of a CU, and whether after a prefix
    got = {i[:5] for i in instances(q.LIB_PATH, "attend_kernel") if i[6] == after_prefix}
    if after_prefix:  # at D = 256 in a launch of its own, else in one with the common tokens
        got |= instances(q.LIB_PATH, "shared_kernel")
    assert got == want
